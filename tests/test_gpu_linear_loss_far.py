"""The linear head's cross entropy and its gradient with infinities: in dloss.  Bounds: linear_cases.py."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg
from tests.linear_cases import BF16, DEV, FP16, check_loss_grad, loss64, loss_inputs, randn

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
INF = float("inf")


def nan(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


@DTYPES
@pytest.mark.parametrize("others", [20.0, 1e-5])
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
def test_a_dloss_that_is_no_number_stays_in_its_row(dtype, others, bad):
    """dx of the other rows is what it is without that row, whichever size their dloss has."""
    rows, width, vocab = 60, 72, 300
    x, w, target = loss_inputs(rows, width, vocab, dtype, 41, ignored=0.0)
    lse = loss64(x, w, target)[1].float()
    dloss = randn(1, rows, scale=others)
    dloss[5] = 0.0
    want, dx = nan(rows, width, dtype=dtype), nan(rows, width, dtype=dtype)
    tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, want)
    check_loss_grad(dloss, x, w, target, lse, want, None, "finite")
    dloss[5] = bad
    dw = nan(vocab, width, dtype=dtype)
    tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, dx, dw)
    assert not torch.isfinite(dx[5]).any() and not torch.isfinite(dw[target[5]]).any()
    rest = torch.arange(rows, device=DEV) != 5
    assert torch.equal(dx[rest], want[rest])
