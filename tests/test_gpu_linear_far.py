"""The gated projection and its gradient where a projection is far out: past 2^64, whose
square fp32 does not hold, and infinite.  Bounds: linear_cases.py."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg
from tests.linear_cases import ACTS, BF16, DEV, FP16, act64, check_gated_grad, gated_inputs, half, randn

pytestmark = pytest.mark.gpu

FAR = [0.0, 1.0, -1.0, 50.0, -50.0, 1e4, -1e4, 2.0 ** 63, 2.0 ** 64, -(2.0 ** 64), 2.0 ** 65, 1e20, -1e20, 1e30, -1e30, 3e38, -3e38]


def same(got, want, bound, what):
    """NaN and infinities where `want` has them, within `bound` elsewhere."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    far = torch.isinf(want)
    assert torch.equal(got[far], want[far]), what
    there = torch.isfinite(want)
    assert torch.isfinite(got[there]).all(), what
    assert ((got - want).abs()[there] <= bound[there]).all(), what


# both forms of the kernel for few rows, both tiles, a tile cut and a whole one
@pytest.mark.parametrize("rows,width,hidden", [(16, 8, 40), (32, 72, 40), (40, 72, 33), (300, 8, 256), (2048, 64, 4096)])
@pytest.mark.parametrize("act", ACTS)
def test_far_projections(act, rows, width, hidden):
    """g = a c and u = b, exactly: x = (a, 1, 0 ...), the weights' rows (c, 0 ...) and (0, b, 0 ...).
    y is off by its rounding and the activation's 2^-17 |y| + 2^-22 |u|.  act(inf) is inf; act(-inf)
    is NaN, as -inf times 0 is."""
    a = torch.tensor(FAR, device=DEV).repeat(rows // len(FAR) + 1)[:rows].to(BF16)
    c = torch.tensor([1.0, -1.0, 4.0], device=DEV).repeat(hidden // 3 + 1)[:hidden].to(BF16)
    b = torch.tensor([1.0, -0.5], device=DEV).repeat(hidden // 2 + 1)[:hidden].to(BF16)
    x, wg, wu = (torch.zeros((n, width), dtype=BF16, device=DEV) for n in (rows, hidden, hidden))
    x[:, 0], x[:, 1], wg[:, 0], wu[:, 1] = a, 1.0, c, b
    y, gate, up = (torch.full((rows, hidden), float("nan"), dtype=BF16, device=DEV) for _ in range(3))
    tsg.gated_linear(x, wg, wu, y, act, gate=gate, up=up)
    g, u = (a.float()[:, None] * c.float()[None]).double(), b.double()[None].expand(rows, hidden)
    assert torch.isinf(g).any() and torch.equal(gate.double(), g) and torch.equal(up.double(), u)
    want = act64(act, g)[0] * u
    same(y, want, (half(BF16) + 2.0 ** -17) * want.abs() + 2.0 ** -22 * u.abs(), act)


@pytest.mark.parametrize("act", ACTS)
def test_far_gates(act):
    """The slopes end in 0 and 1, and a far gate reaches nothing but its own sums."""
    rows, width, hidden = 40, 64, 70
    x, wg, wu = gated_inputs(rows, width, hidden, BF16, 31)
    dy, gate, up = randn(1, rows, hidden).to(BF16), randn(2, rows, hidden, scale=2).to(BF16), randn(3, rows, hidden).to(BF16)
    for i, g in enumerate((-(2.0 ** 64), -1e20, -1e30, -3e38, 2.0 ** 64, 1e20)):
        gate[3 * i, 5 * i] = g
    dx, dwg, dwu = (torch.full(t.shape, float("nan"), dtype=BF16, device=DEV) for t in (x, wg, wu))
    tsg.gated_linear_grad(dy, x, wg, wu, gate, up, dx, dwg, dwu, act)
    check_gated_grad(dy, x, wg, wu, gate, up, act, dx, dwg, dwu, "far gates")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_infinite_gates(dtype, act):
    """An infinite gate, which fp16 keeps of a g from 65520 on, stands for a far one: act(-inf) is 0,
    the slopes are 0 and 1.  The same bits as from gates of 1e4 to either side, where act and slope
    have ended, but for the sums that hold dy act(inf)."""
    rows, width, hidden = 40, 64, 70
    x, wg, wu = gated_inputs(rows, width, hidden, dtype, 32)
    dy, gate, up = randn(1, rows, hidden).to(dtype), randn(2, rows, hidden, scale=2).to(dtype), randn(3, rows, hidden).to(dtype)
    near = gate.clone()
    for at, g in (((3, 5), -1.0), ((8, 5), -1.0), ((9, 69), -1.0), ((7, 9), 1.0)):
        gate[at], near[at] = g * float("inf"), g * 1e4
    got, want = ([torch.full(t.shape, float("nan"), dtype=dtype, device=DEV) for t in (x, wg, wu)] for _ in range(2))
    tsg.gated_linear_grad(dy, x, wg, wu, gate, up, *got, act)
    tsg.gated_linear_grad(dy, x, wg, wu, near, up, *want, act)
    check_gated_grad(dy, x, wg, wu, near, up, act, *want, "near")
    assert torch.equal(got[1], want[1])
    for i, at in ((0, 7), (2, 9)):
        assert not torch.isfinite(got[i][at]).any()
        got[i][at] = want[i][at]
        assert torch.equal(got[i], want[i])
