"""Views into one buffer: matrices that lie between each other's rows are not
overlapping, and every call takes them; a call in place is refused and changes
nothing."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _packed(rows, width, parts, dtype):
    g = torch.Generator().manual_seed(rows + width)
    big = torch.randn((rows, parts * width), generator=g).to(dtype).to(DEV)
    return big, [big[:, i * width:(i + 1) * width] for i in range(parts)]


@pytest.mark.parametrize("rows,width", [(1, 64), (40, 96), (300, 2048)])
def test_parts_of_one_buffer(rows, width):
    """x, dy, y, dx and what dequantize writes side by side, the result that of separate tensors."""
    dtype = torch.bfloat16
    big, (x, dy, y, dx, back) = _packed(rows, width, 5, dtype)
    sx, sdy = x.clone(), dy.clone()
    stats, alone = torch.empty((2, rows), device=DEV), torch.empty((2, rows), device=DEV)
    weights = torch.ones((4, width), device=DEV)        # gamma, beta, dgamma, dbeta
    apart = torch.ones((4, width), device=DEV)
    codes, scales = (torch.empty((rows, n), dtype=torch.uint8, device=DEV) for n in (width, width // 32))
    sy, sdx, sback = (torch.empty((rows, width), dtype=dtype, device=DEV) for _ in range(3))
    for a, b, c, d, e, s, w in ((x, dy, y, dx, back, stats, weights), (sx, sdy, sy, sdx, sback, alone, apart)):
        for kw in ({}, {"stream": torch.cuda.current_stream()}):
            tsg.layer_norm(a, w[0], w[1], 1e-5, y=c, mean=s[0], rstd=s[1])
            tsg.layer_norm_grad(b, a, w[0], s[0], s[1], d, w[2], w[3], **kw)
            tsg.mx_quantize(c, codes, scales, **kw)
            tsg.mx_dequantize(codes, scales, e, **kw)
    for a, b in ((x, sx), (dy, sdy), (y, sy), (dx, sdx), (back, sback), (stats, alone), (weights, apart)):
        assert torch.equal(a, b)


def test_in_place_is_refused():
    rows, width = 64, 128
    _, (x, dy) = _packed(rows, width, 2, torch.bfloat16)
    x, dy = x.clone(), dy.clone()
    kept, kept_dy = x.clone(), dy.clone()
    v, r = torch.ones(width, device=DEV), torch.ones(rows, device=DEV)
    for kw in ({}, {"stream": torch.cuda.current_stream()}):
        with pytest.raises(tsg.TsgemmError, match="y overlaps x"):
            tsg.layer_norm(x, v, v, 1e-5, y=x, **kw)
        with pytest.raises(tsg.TsgemmError, match="dx overlaps dy"):
            tsg.layer_norm_grad(dy, x, v, r, r, dy, v.clone(), v.clone(), **kw)
        with pytest.raises(tsg.TsgemmError, match="dx overlaps x"):
            tsg.layer_norm_grad(dy, x, v, r, r, x, **kw)
        with pytest.raises(tsg.TsgemmError, match="codes overlaps x"):
            tsg.mx_quantize(x, x.view(torch.uint8).view(-1)[: rows * width].view(rows, width),
                            torch.empty((rows, width // 32), dtype=torch.uint8, device=DEV), **kw)
    torch.cuda.synchronize()
    assert torch.equal(x, kept) and torch.equal(dy, kept_dy)
