"""The gated projection, the cross entropy of a linear head and their gradients on
the GPU against plain fp64 formulas, within the bounds that linear_cases.py derives."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg
from tests.linear_cases import (ACTS, BF16, DEV, FP16, act64, check, check_gated, check_gated_grad, check_loss, check_loss_grad,
                                gated_inputs, loss64, loss_inputs, randn)

pytestmark = pytest.mark.gpu

# rows, width, hidden: one value, tiles' borders, odd ones, several tiles
GATED = [(1, 8, 1), (1, 64, 7), (2, 4096, 130), (3, 72, 33), (16, 136, 64), (17, 128, 129), (63, 200, 65), (128, 64, 64), (129, 264, 257),
         (255, 512, 300), (256, 256, 256), (300, 520, 641)]
# few rows, more weight rows than the workgroups take at a time
GATED_FEW = [(1, 72, 8300), (16, 1032, 9001), (17, 520, 8200), (32, 4104, 64), (33, 4104, 64)]
# ... with tiles of 256
GATED_LARGE = [(2048, 64, 4096), (2049, 200, 4097)]


def nan(rows, width, dtype):
    return torch.full((rows, width), float("nan"), dtype=dtype, device=DEV)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_gated_linear(dtype, act):
    for rows, width, hidden in GATED + GATED_FEW:
        x, wg, wu = gated_inputs(rows, width, hidden, dtype, rows + hidden)
        y, gate, up = (nan(rows, hidden, dtype) for _ in range(3))
        tsg.gated_linear(x, wg, wu, y, act, gate=gate, up=up)
        check_gated(x, wg, wu, act, y, gate, up, f"{rows}x{width}x{hidden}")
        z = nan(rows, hidden, dtype)
        tsg.gated_linear(x, wg, wu, z, act)
        assert torch.equal(y, z)


@pytest.mark.parametrize("rows,width,hidden", GATED_LARGE)
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_gated_linear_large_tiles(dtype, rows, width, hidden):
    x, wg, wu = gated_inputs(rows, width, hidden, dtype, 5)
    y, gate, up = (nan(rows, hidden, dtype) for _ in range(3))
    tsg.gated_linear(x, wg, wu, y, "silu", gate=gate, up=up)
    check_gated(x, wg, wu, "silu", y, gate, up, "large")


def grads(rows, width, hidden, dtype):
    return nan(rows, width, dtype), nan(hidden, width, dtype), nan(hidden, width, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_gated_linear_grad(dtype, act):
    for rows, width, hidden in GATED:
        x, wg, wu = gated_inputs(rows, width, hidden, dtype, rows + hidden)
        gate, up, dy = randn(1, rows, hidden, scale=2).to(dtype), randn(2, rows, hidden).to(dtype), randn(3, rows, hidden, scale=0.1).to(dtype)
        dx, dwg, dwu = grads(rows, width, hidden, dtype)
        tsg.gated_linear_grad(dy, x, wg, wu, gate, up, dx, dwg, dwu, act)
        check_gated_grad(dy, x, wg, wu, gate, up, act, dx, dwg, dwu, f"{rows}x{width}x{hidden}")
        ex, eg, eu = grads(rows, width, hidden, dtype)
        tsg.gated_linear_grad(dy, x, wg, wu, gate, up, dx=ex, act=act)
        tsg.gated_linear_grad(dy, x, wg, wu, gate, up, dgate_weight=eg, dup_weight=eu, act=act)
        assert torch.equal(dx, ex) and torch.equal(dwg, eg) and torch.equal(dwu, eu)


@pytest.mark.parametrize("rows,width,hidden", [(2048, 2048, 4100), (4100, 1032, 1100), (30000, 136, 300)])
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_gated_linear_grad_large_and_split(dtype, rows, width, hidden):
    x, wg, wu = gated_inputs(rows, width, hidden, dtype, 6)
    gate, up, dy = randn(1, rows, hidden, scale=2).to(dtype), randn(2, rows, hidden).to(dtype), randn(3, rows, hidden, scale=0.1).to(dtype)
    dx, dwg, dwu = grads(rows, width, hidden, dtype)
    tsg.gated_linear_grad(dy, x, wg, wu, gate, up, dx, dwg, dwu)
    check_gated_grad(dy, x, wg, wu, gate, up, "silu", dx, dwg, dwu, "large")


# rows, width, vocab
LOSS = [(1, 8, 1), (1, 64, 2), (2, 72, 33), (1, 2048, 1000), (16, 136, 127), (17, 128, 128), (63, 200, 129), (128, 64, 640), (129, 264, 257),
        (255, 512, 1000), (256, 256, 512), (300, 520, 5003)]


@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_linear_cross_entropy(dtype):
    for rows, width, vocab in LOSS + [(2049, 72, 8200), (3, 72, 20000), (16, 1032, 9001), (17, 136, 8200), (32, 4104, 64), (33, 4104, 64)]:
        x, w, target = loss_inputs(rows, width, vocab, dtype, rows + vocab)
        loss, lse = (torch.full((rows,), float("nan"), device=DEV) for _ in range(2))
        tsg.linear_cross_entropy(x, w, target, loss, lse)
        check_loss(x, w, target, loss, lse, f"{rows}x{width}x{vocab}")


@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_linear_cross_entropy_grad(dtype):
    for rows, width, vocab in LOSS:
        x, w, target = loss_inputs(rows, width, vocab, dtype, rows + vocab)
        lse = loss64(x, w, target)[1].float()
        dloss = randn(9, rows, scale=0.3)
        dx, dw = nan(rows, width, dtype), nan(vocab, width, dtype)
        tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, dx, dw)
        check_loss_grad(dloss, x, w, target, lse, dx, dw, f"{rows}x{width}x{vocab}")
        ex, ew = nan(rows, width, dtype), nan(vocab, width, dtype)
        tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, dx=ex)
        tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, dweight=ew)
        assert torch.equal(dx, ex) and torch.equal(dw, ew)


# tiles of 256 and splits; several pieces of the vocabulary
@pytest.mark.parametrize("rows,width,vocab", [(2049, 1032, 9000), (20000, 64, 15001), (5000, 520, 60000)])
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_linear_cross_entropy_grad_large_and_pieces(dtype, rows, width, vocab):
    x, w, target = loss_inputs(rows, width, vocab, dtype, 7)
    lse = loss64(x, w, target)[1].float()
    dloss = torch.full((rows,), 1.0 / rows, device=DEV)
    dx, dw = nan(rows, width, dtype), nan(vocab, width, dtype)
    if dtype == FP16:
        dloss *= 1024
    tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, dx, dw)
    check_loss_grad(dloss, x, w, target, lse, dx, dw, "large")
