"""The wait states around the MFMAs and LDS-DMAs of the linear layers' tile kernel,
which sit in inline asm that the compiler does not look into: the rules and the
search along every path are those of test_wgrad_operand_hazards.py.  Compiles the
kernels to assembly (no GPU); with TSGEMM_STRESS_TEST=1 those of the race-detection
build too."""

import os
import subprocess

import pytest

from persistent_tile_scheduled_amd import _build
from tests.test_wgrad_operand_hazards import hazards


@pytest.mark.parametrize("stress", [0, 1])
@pytest.mark.parametrize("dtype", [1, 2])
def test_every_path_keeps_the_wait_states(tmp_path, dtype, stress):
    if stress and os.environ.get("TSGEMM_STRESS_TEST") != "1":
        pytest.skip("the race-detection build is looked at with TSGEMM_STRESS_TEST=1")
    out = os.path.join(tmp_path, "linear.s")
    flags = [f for f in _build.FLAGS if f != "-fPIC"]
    r = subprocess.run([_build.HIPCC] + flags + [f"-DTSG_STRESS={stress}", f"-DTSG_LIN_DT={dtype}", "--cuda-device-only", "-S",
                                                 os.path.join(_build.CSRC, "tsgemm_linear_tu.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        asm = f.read()
    assert "_ZN3tsg13linear_kernel" in asm
    found = hazards(asm.replace("_ZN3tsg13linear_kernel", "_ZN3tsg12wgrad_kernel"))  # the search goes by the name
    assert len(found) == 10, sorted(found)
    assert not any(found.values()), {k: (len(v), v[:3]) for k, v in found.items() if v}
