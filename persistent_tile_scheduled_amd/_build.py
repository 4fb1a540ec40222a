"""Build step for libtsgemm.so (hipcc, gfx950), kept beside the sources it builds.

The kernels are split over translation units that compile in parallel: the
host code (tsgemm.hip), one unit per fp16/bf16 dtype and tile shape
(tsgemm_gemm_tu.hip with -DTSG_TU_*), the block-scaled FP8 unit
(tsgemm_mx_tu.hip), and the operators around it: their host code
(tsgemm_ops.hip), the row operators (tsgemm_rows_tu.hip) and the weight
gradient (tsgemm_wgrad_tu.hip); the gated projection and the linear head's cross
entropy: their host code (tsgemm_linear.hip) and one unit per type
(tsgemm_linear_tu.hip with -DTSG_LIN_DT).  The objects are linked into one shared library.
Beside it lies the binding's extension module (tsgemm_torch.cpp, g++ and torch's
headers), which holds no kernel.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libtsgemm.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 VALU ops are kept off in every HIP build of this project
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]

# (source, extra defines, object name)
GEMM_TUS = [(dt, bm, bk) for dt in (1, 2) for bm in (128, 256) for bk in (32, 64)]
UNITS = ([("tsgemm.hip", [], "host.o"), ("tsgemm_mx_tu.hip", [], "mx.o"),
          ("tsgemm_ops.hip", [], "ops.o"), ("tsgemm_rows_tu.hip", [], "rows.o"),
          ("tsgemm_wgrad_tu.hip", [], "wgrad.o"), ("tsgemm_linear.hip", [], "linear.o")] +
         [("tsgemm_linear_tu.hip", [f"-DTSG_LIN_DT={dt}"], f"linear_{dt}.o") for dt in (1, 2)] +
         [("tsgemm_gemm_tu.hip", [f"-DTSG_TU_DT={dt}", f"-DTSG_TU_BM={bm}", f"-DTSG_TU_BK={bk}"],
           f"gemm_{dt}_{bm}_{bk}.o") for dt, bm, bk in GEMM_TUS])


TORCH_OUT = os.path.join(HERE, "_tsgemm_torch.so")


def build_torch_module(out: str = TORCH_OUT) -> str:
    """Compile the binding's extension module at `out`."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = out + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"]]
    for d in cpp_extension.include_paths():
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "tsgemm_torch.cpp"), "-o", tmp, "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10",
            f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on tsgemm_torch.cpp:\n" + r.stderr[-4000:])
    os.replace(tmp, out)
    return out


def _jobs() -> int:
    n = os.cpu_count() or 4
    cap = int(os.environ.get("MAX_JOBS", "16"))
    return max(1, min(n, cap, len(UNITS)))


STRESS_OUT = os.path.join(HERE, "libtsgemm_stress.so")


def build_stress_library(out: str = STRESS_OUT) -> str:
    """The race-detection build (-DTSG_STRESS=1: random pauses at every barrier
    and DMA).  Tests run against it with TSGEMM_LIB=<this file>."""
    return build_library(out=out, extra_flags=["-DTSG_STRESS=1"])


def build_library(out: str = OUT, verbose: bool = False, extra_flags=()) -> str:
    """Compile every unit (in parallel) and link libtsgemm.so at `out`.
    `extra_flags` are added to every compile (e.g. -D switches of a variant build)."""
    tmpdir = tempfile.mkdtemp(prefix="tsgemm_build_")
    try:
        def compile_one(unit):
            src, defs, obj = unit
            cmd = [HIPCC] + FLAGS + list(extra_flags) + defs + ["-c", os.path.join(CSRC, src),
                                                                "-o", os.path.join(tmpdir, obj)]
            r = subprocess.run(cmd, capture_output=True, text=True)
            return unit, r

        with concurrent.futures.ThreadPoolExecutor(_jobs()) as ex:
            results = list(ex.map(compile_one, UNITS))
        for (src, defs, _), r in results:
            if r.returncode != 0:
                raise RuntimeError(f"hipcc failed on {src} {' '.join(defs)}:\n" + r.stderr[-4000:])
            if verbose and r.stderr:
                print(r.stderr[-2000:])
        tmp = out + ".tmp%d" % os.getpid()
        cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC"] + \
            [os.path.join(tmpdir, obj) for _, _, obj in UNITS] + ["-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stderr[-4000:])
        os.replace(tmp, out)
    finally:
        shutil.rmtree(tmpdir, ignore_errors=True)
    return out


def main(argv) -> None:
    """What the package loads, or with --stress the race-detection library."""
    if "--stress" in argv:
        print(build_stress_library())
    else:
        print(build_library())
        print(build_torch_module())


if __name__ == "__main__":
    import sys
    main(sys.argv[1:])
