"""The linear head's cross entropy for more rows than one launch may have threads over 64."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg
from tests.linear_cases import BF16, DEV, U

pytestmark = pytest.mark.gpu


def test_more_rows_than_a_join_has_groups():
    """2^26 + 5 rows, in fp64 a stretch at a time.  The logits' sums have 8 terms, all below 2^6."""
    rows, width, vocab = (1 << 26) + 5, 8, 9
    g = torch.Generator(device=DEV)
    g.manual_seed(51)
    x = torch.empty((rows, width), dtype=BF16, device=DEV)
    for i in range(0, rows, 1 << 23):
        x[i: i + (1 << 23)] = torch.randn(x[i: i + (1 << 23)].shape, generator=g, device=DEV)
    w = torch.randn((vocab, width), generator=g, device=DEV).to(BF16)
    target = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    loss, lse = (torch.full((rows,), float("nan"), device=DEV) for _ in range(2))
    tsg.linear_cross_entropy(x, w, target, loss, lse)
    for i in range(0, rows, 1 << 22):
        s = slice(i, min(i + (1 << 22), rows))
        l = x[s].double() @ w.double().t()
        assert l.abs().max() < 2.0 ** 6
        want = torch.logsumexp(l, dim=1)
        # 2 K u sum|terms| below 2^-14 for the logits, 2^-17 and 2^-21 max|l| for the exponentials' sum
        off = 2.0 ** -14 + 2.0 ** -17 + 2.0 ** -15 + U * 2.0 ** 6
        assert ((lse[s] - want).abs() <= off).all() and torch.isfinite(lse[s]).all()
        hit = l.gather(1, target[s, None])[:, 0]
        assert ((loss[s] - (want - hit)).abs() <= 2 * off).all() and torch.isfinite(loss[s]).all()
    del x
    torch.cuda.empty_cache()
