"""The linear head's cross entropy and its gradient with infinities in dloss and in
single logits, and with logits as far out as fp32 goes.  Bounds: linear_cases.py."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg
from tests.linear_cases import BF16, DEV, FP16, U, check_loss, check_loss_grad, half, loss64, loss_inputs, randn

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


@DTYPES
@pytest.mark.parametrize("rows", [16, 30, 100, 600])
def test_infinite_logits(dtype, rows):
    """x[:, 0] is 1, so a weight of -inf there is a logit of -inf: its exponential is 0 and the row
    is that of the other words; the loss of such a target is inf.  A logit of inf makes a row NaN, a
    row of nothing but -inf has an lse of -inf and no loss."""
    width, vocab = 64, 515
    x, w, target = loss_inputs(rows, width, vocab, dtype, 43, ignored=0.1)
    x[:, 0] = 1.0
    out = torch.arange(vocab, device=DEV) % 3 == 1
    w[out, 0] = -INF
    keep = torch.nonzero(~out)[:, 0]
    at = torch.full((vocab,), -7, device=DEV)      # of no word that is left
    at[keep] = torch.arange(len(keep), device=DEV)
    counted = target != -100
    gone = counted & out[target.clamp_min(0)]
    assert gone.any() and (counted & ~gone).any()
    moved = torch.where(counted & ~gone, at[target.clamp_min(0)], -100)
    loss, lse = nan(rows), nan(rows)
    tsg.linear_cross_entropy(x, w, target, loss, lse)
    assert (loss[gone] == INF).all()
    check_loss(x, w[keep], moved, torch.where(gone, 0.0, loss), lse, "-inf here and there")
    dloss, dw = torch.where(gone, 0.0, randn(1, rows)), nan(vocab, width, dtype=dtype)
    masked = torch.where(gone, -100, target)
    tsg.linear_cross_entropy_grad(dloss, x, w, masked, lse, dweight=dw)
    check_loss_grad(dloss, x, w[keep], moved, lse, None, dw[keep], "-inf here and there")
    assert not dw[out].any()
    x[3, 0] = -1.0                                  # ... of inf
    tsg.linear_cross_entropy(x, w, target, loss, lse)
    assert torch.isnan(lse[3]) and (torch.isnan(loss[3]) if counted[3] else loss[3] == 0) and torch.isfinite(lse).sum() == rows - 1
    x[3, 0] = 1.0
    w[:, 0] = -INF
    tsg.linear_cross_entropy(x, w, target, loss, lse)
    assert (lse == -INF).all() and torch.isnan(loss[counted]).all() and not loss[~counted].any()


# type, x[:, 0] and the size of w[:, 0]: logits of up to their product, all of one sign or of both
FAR = [(FP16, 1.0, 6e4), (FP16, 6e4, 6e4), (BF16, 1.0, 1e5), (BF16, 1.0, 1e9), (BF16, 1.0, 1e12), (BF16, 1.0, 1e30), (BF16, 1.0, 3e38)]


def far_logits(dtype, x0, size, signs, rows, vocab):
    """Exact logits x0 w[:, 0] (the other values are zeros), the two largest of them alike."""
    x, w = torch.zeros((rows, 8), dtype=dtype, device=DEV), torch.zeros((vocab, 8), dtype=dtype, device=DEV)
    v = size * (0.1 + 0.9 * torch.rand(vocab, generator=torch.Generator().manual_seed(7)).to(DEV))
    w[:, 0] = {"+": 1, "-": -1, "+-": 1 - 2 * (torch.arange(vocab, device=DEV) % 2)}[signs] * v
    top = w[:, 0].argmax()
    w[(top + 2) % vocab] = w[top]
    x[:, 0] = x0
    target = torch.arange(rows, device=DEV) * 37 % vocab
    target[::3] = top
    return x, w, target


@pytest.mark.parametrize("signs", ["+", "-", "+-"])
@pytest.mark.parametrize("rows", [5, 30, 100, 600])
def test_far_logits(rows, signs):
    """lse is off by its exponentials' sum, 2^-17, and its rounding; the gradient, which goes by that
    lse, by 2^-18 p, its rounding of dl and the sums'.  Apart from those, what is below 2^-126, the least
    normal value of fp32 and bf16, may be 0: exp of a difference past -88 is.  The sums are formed over
    the largest |dloss|, 0.25, and multiplied with it afterwards: where their terms over it pass fp32's
    3.4e38 (weights of 3e38 alone) dx may be infinite."""
    vocab = 515
    for dtype, x0, size in FAR:
        x, w, target = far_logits(dtype, x0, size, signs, rows, vocab)
        l = x.double() @ w.double().t()
        want, hit = torch.logsumexp(l, dim=1), l.gather(1, target[:, None])[:, 0]
        loss, lse = nan(rows), nan(rows)
        tsg.linear_cross_entropy(x, w, target, loss, lse)
        assert torch.isfinite(lse).all(), (dtype, x0, size)
        assert ((lse - want).abs() <= 2.0 ** -17 + 2 * U * want.abs()).all(), (dtype, x0, size)
        fits = want - hit < 3e38
        assert ((loss - (want - hit)).abs() <= 2.0 ** -17 + 2 * U * (want - hit).abs())[fits].all(), (dtype, x0, size)
        e, dloss = half(dtype), torch.full((rows,), 0.25, device=DEV)
        dx, dw = nan(rows, 8, dtype=dtype), nan(vocab, 8, dtype=dtype)
        tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, dx, dw)
        p = torch.exp(l - lse.double()[:, None])
        dl = 0.25 * p
        off = 2.0 ** -20 * p
        dl[torch.arange(rows, device=DEV), target] -= 0.25
        off = off + (e + 2.0 ** -20) * dl.abs() + (2.0 ** -39 if dtype == FP16 else 2.0 ** -126)
        tiny = 2.0 ** -25 if dtype == FP16 else 2.0 ** -126
        for got, a, b in ((dx, (dl, off), w.double()), (dw, (dl.t(), off.t()), x.double())):
            ref = a[0] @ b
            bound = e * ref.abs() + (a[1] + 2 * (a[0].shape[1] + 64) * U * a[0].abs()) @ b.abs() + tiny
            there = (ref.abs() < 0.99 * torch.finfo(dtype).max) & (a[0].abs() @ b.abs() / 0.25 < 3.4e38)
            assert ((got - ref).abs() <= bound)[there].all(), (dtype, x0, size)
