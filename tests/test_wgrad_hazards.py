"""The weight gradient's MFMAs sit in inline asm, whose results the compiler does
not know to wait for: an accumulator that it copies, spills or stores too soon
after the MFMA that writes it would be read stale.  Compiles the kernels to
assembly (under a minute, no GPU) and looks for such accesses; with
TSGEMM_STRESS_TEST=1 those of the race-detection build too."""

import os
import re
import subprocess

from persistent_tile_scheduled_amd import _build

# a 16x16x32 MFMA's result -> any other instruction's access: 8 wait states
NEAR = 9


def _accumulators(text):
    out = set()
    for a, b in re.findall(r"\ba\[(\d+):(\d+)\]", text):
        out |= set(range(int(a), int(b) + 1))
    return out | {int(a) for a in re.findall(r"\ba(\d+)\b", text)}


def near_accesses(asm):
    """{kernel: accesses of an accumulator within NEAR wait states of the MFMA
    before it that wrote it}, code taken in the order it lies in."""
    found = {}
    for name, body in re.findall(r"^(_ZN3tsg12wgrad_kernel\w+):.*?\n(.*?)\n\s*s_endpgm", asm, re.S | re.M):
        at, written, found[name] = 0, [], []
        for line in map(str.strip, body.split("\n")):
            if not line or line[0] in ";.":
                continue
            op = line.split()[0]
            at += int(line.split()[1]) + 1 if op == "s_nop" else 1
            if op.startswith("v_mfma"):
                written = written[-NEAR:] + [(at, _accumulators(line[len(op):].split(",")[0] + "," + line.split(",")[0]))]
                continue
            used = _accumulators(line)
            if used and any(at - when < NEAR and used & regs for when, regs in written):
                found[name].append(line)
    return found


def test_the_search_finds_a_planted_access():
    asm = "_ZN3tsg12wgrad_kernelX: ;\n v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n%s v_accvgpr_read_b32 v9, a2\n s_endpgm\n"
    assert near_accesses(asm % "")["_ZN3tsg12wgrad_kernelX"] == ["v_accvgpr_read_b32 v9, a2"]
    assert near_accesses(asm % " s_nop 7\n s_nop 0\n")["_ZN3tsg12wgrad_kernelX"] == []


def _compiled(tmp_path, stress):
    out = os.path.join(tmp_path, f"wgrad{stress}.s")
    flags = [f for f in _build.FLAGS if f != "-fPIC"]
    r = subprocess.run([_build.HIPCC] + flags + [f"-DTSG_STRESS={stress}", "--cuda-device-only", "-S",
                                                 os.path.join(_build.CSRC, "tsgemm_wgrad_tu.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        return f.read()


def test_no_accumulator_is_touched_right_after_its_mfma(tmp_path):
    for stress in (0, 1) if os.environ.get("TSGEMM_STRESS_TEST") == "1" else (0,):
        found = near_accesses(_compiled(tmp_path, stress))
        assert len(found) == 8, sorted(found)
        assert not any(found.values()), {k: v[:3] for k, v in found.items() if v}
