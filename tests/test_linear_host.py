"""Refusals, workspaces and empty calls of the gated projection and of the linear
head's cross entropy, without a GPU: the checks come before any launch."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg

# addresses far from each other that nothing reads
P = {name: (i + 1) << 40 for i, name in enumerate(
    "x wg wu y gate up dy dx dwg dwu ws w target loss lse dloss dw".split())}


def _gated(rows=4, hidden=24, width=64, dt=2, act=1, ldx=64, ldgw=64, lduw=64, ldy=24, ldgate=24, ldup=24, stream=None, **p):
    p = {**P, **p}
    return tsg.load().tsgemm_gated_linear(rows, hidden, width, dt, act, p["x"], ldx, p["wg"], ldgw, p["wu"], lduw, p["y"], ldy,
                                          p["gate"], ldgate, p["up"], ldup, stream)


def _gated_grad(rows=4, hidden=24, width=64, dt=2, act=1, lddy=24, ldx=64, ldgw=64, lduw=64, ldgate=24, ldup=24, lddx=64, lddgw=64,
                ldduw=64, size=1 << 30, stream=None, **p):
    p = {**P, **p}
    return tsg.load().tsgemm_gated_linear_grad(rows, hidden, width, dt, act, p["dy"], lddy, p["x"], ldx, p["wg"], ldgw, p["wu"], lduw,
                                               p["gate"], ldgate, p["up"], ldup, p["dx"], lddx, p["dwg"], lddgw, p["dwu"], ldduw,
                                               p["ws"], size, stream)


def _loss(rows=4, vocab=24, width=64, dt=2, ldx=64, ldw=64, ignore=-100, size=1 << 30, stream=None, **p):
    p = {**P, **p}
    return tsg.load().tsgemm_linear_cross_entropy(rows, vocab, width, dt, p["x"], ldx, p["w"], ldw, p["target"], ignore, p["loss"],
                                                  p["lse"], p["ws"], size, stream)


def _loss_grad(rows=4, vocab=24, width=64, dt=2, ldx=64, ldw=64, ignore=-100, lddx=64, lddw=64, size=1 << 30, stream=None, **p):
    p = {**P, **p}
    return tsg.load().tsgemm_linear_cross_entropy_grad(rows, vocab, width, dt, p["dloss"], p["x"], ldx, p["w"], ldw, p["target"], ignore,
                                                       p["lse"], p["dx"], lddx, p["dw"], lddw, p["ws"], size, stream)


COMMON = [
    (dict(rows=-1), tsg.EINVAL, "rows"), (dict(rows=1 << 31), tsg.EINVAL, "2^31"), (dict(width=0), tsg.EINVAL, "multiple of 8"),
    (dict(width=63), tsg.EINVAL, "multiple of 8"), (dict(width=1 << 23, ldx=1 << 23), tsg.EUNSUPPORTED, "2^23"),
    (dict(dt=4), tsg.EINVAL, "dtype"), (dict(dt=3), tsg.EINVAL, "dtype"), (dict(x=None), tsg.EINVAL, "x is NULL"),
    (dict(x=P["x"] + 8), tsg.EINVAL, "rows of x"), (dict(x=P["x"] + 1), tsg.EINVAL, "x must be aligned"), (dict(ldx=56), tsg.EINVAL, "row stride of x"),
    (dict(ldx=68), tsg.EINVAL, "rows of x"), (dict(ldx=1 << 23), tsg.EUNSUPPORTED, "row stride of x"),
    (dict(rows=1 << 30, width=1 << 12, ldx=1 << 12), tsg.EUNSUPPORTED, "2^40"),
]
WORK = [(dict(ws=None), tsg.EINVAL, "workspace"), (dict(ws=P["ws"] + 8), tsg.EINVAL, "workspace"), (dict(size=0), tsg.EINVAL, "workspace")]


def refused(call, kw, code, needle):
    assert call(**kw) == code
    assert needle in tsg.last_error(), tsg.last_error()
    assert tsg.load().tsgemm_last_error_code() == code


@pytest.mark.parametrize("kw,code,needle", COMMON + [
    (dict(hidden=-1), tsg.EINVAL, "hidden"), (dict(hidden=1 << 30), tsg.EUNSUPPORTED, "hidden"), (dict(act=0), tsg.EINVAL, "act"),
    (dict(act=4), tsg.EINVAL, "act"), (dict(wg=None), tsg.EINVAL, "gate_weight is NULL"), (dict(wu=P["wu"] + 2), tsg.EINVAL, "rows of up_weight"),
    (dict(ldgw=60), tsg.EINVAL, "gate_weight"), (dict(lduw=66), tsg.EINVAL, "up_weight"), (dict(y=None), tsg.EINVAL, "y is NULL"),
    (dict(ldy=23), tsg.EINVAL, "row stride of y"), (dict(y=P["y"] + 1), tsg.EINVAL, "y must be aligned"), (dict(ldgate=20), tsg.EINVAL, "row stride of gate"),
    (dict(y=P["x"]), tsg.EINVAL, "y overlaps x"), (dict(gate=P["y"] + 2), tsg.EINVAL, "gate overlaps y"),
    (dict(up=P["wu"] + 64), tsg.EINVAL, "up overlaps up_weight"),
])
def test_gated_linear_refuses(kw, code, needle):
    refused(_gated, kw, code, needle)


@pytest.mark.parametrize("kw,code,needle", COMMON + WORK + [
    (dict(hidden=1 << 22), tsg.EUNSUPPORTED, "2^22"), (dict(act=9), tsg.EINVAL, "act"), (dict(dwg=None), tsg.EINVAL, "together"),
    (dict(dwu=None), tsg.EINVAL, "together"), (dict(dx=None, dwg=None, dwu=None), tsg.EINVAL, "no output"), (dict(gate=None), tsg.EINVAL, "gate is NULL"),
    (dict(up=None), tsg.EINVAL, "up is NULL"), (dict(dy=None), tsg.EINVAL, "dy is NULL"), (dict(lddx=60), tsg.EINVAL, "dx"),
    (dict(dwg=P["dwg"] + 2), tsg.EINVAL, "rows of dgate_weight"), (dict(ldduw=72 + 4), tsg.EINVAL, "rows of dup_weight"),
    (dict(dx=P["x"]), tsg.EINVAL, "dx overlaps x"), (dict(dwu=P["dwg"]), tsg.EINVAL, "dup_weight overlaps dgate_weight"),
    (dict(ws=P["gate"]), tsg.EINVAL, "workspace overlaps gate"),
])
def test_gated_linear_grad_refuses(kw, code, needle):
    refused(_gated_grad, kw, code, needle)


@pytest.mark.parametrize("kw,code,needle", COMMON + WORK + [
    (dict(vocab=-1), tsg.EINVAL, "vocab"), (dict(vocab=0), tsg.EINVAL, "vocabulary of at least 1"), (dict(vocab=1 << 30), tsg.EUNSUPPORTED, "vocab"),
    (dict(w=None), tsg.EINVAL, "weight is NULL"), (dict(ldw=72 + 4), tsg.EINVAL, "rows of weight"), (dict(target=None), tsg.EINVAL, "target"),
    (dict(target=P["target"] + 4), tsg.EINVAL, "target"), (dict(loss=None), tsg.EINVAL, "loss"), (dict(lse=P["lse"] + 2), tsg.EINVAL, "lse"),
    (dict(lse=P["loss"] + 8), tsg.EINVAL, "lse overlaps loss"), (dict(ws=P["x"] + 64), tsg.EINVAL, "workspace overlaps x"),
])
def test_linear_cross_entropy_refuses(kw, code, needle):
    refused(_loss, kw, code, needle)


@pytest.mark.parametrize("kw,code,needle", COMMON + WORK + [
    (dict(vocab=0), tsg.EINVAL, "vocabulary of at least 1"), (dict(dx=None, dw=None), tsg.EINVAL, "no output"), (dict(dloss=None), tsg.EINVAL, "dloss"),
    (dict(lse=None), tsg.EINVAL, "lse"), (dict(target=None), tsg.EINVAL, "target"), (dict(dw=P["dw"] + 8), tsg.EINVAL, "rows of dweight"),
    (dict(dw=P["w"]), tsg.EINVAL, "dweight overlaps weight"), (dict(dx=P["dw"]), tsg.EINVAL, "dweight overlaps dx"),
    (dict(ws=P["dloss"] - 64), tsg.EINVAL, "workspace overlaps dloss"),
])
def test_linear_cross_entropy_grad_refuses(kw, code, needle):
    refused(_loss_grad, kw, code, needle)


def test_empty_calls_launch_nothing():
    none = dict.fromkeys(P)
    assert _gated(rows=0, **none) == tsg.OK and _gated(hidden=0, **none) == tsg.OK
    assert _loss(rows=0, **none) == tsg.OK
    assert _loss_grad(rows=0, **{**none, "dx": P["dx"]}) == tsg.OK
    assert _gated_grad(rows=0, hidden=0, **{**none, "dx": P["dx"]}) == tsg.OK
    assert tsg.gated_linear_grad_workspace(0, 24, 64) == 0 and tsg.linear_cross_entropy_workspace(0, 24, 64) == 0
    assert tsg.linear_cross_entropy_grad_workspace(0, 24, 64) == 0


def test_workspaces_stay_small():
    """The logits' gradient is held for a piece of the vocabulary: 512 MiB, unless 2048 columns take more."""
    for rows, vocab, width in ((1, 1 << 22, 64), (4096, 1 << 20, 512), (8192, 131072, 4096), (100000, 200000, 64)):
        held = max(512 << 20, 2 * rows * 2048)
        others = 2 * rows * width + 4 * rows * width * 64 + 4 * width * held // (2 * rows) + 32 * rows + 4096
        assert tsg.linear_cross_entropy_grad_workspace(rows, vocab, width) <= held + others
        assert tsg.linear_cross_entropy_workspace(rows, vocab, width) <= 16 * rows * (vocab // 128 + 1) + 4 * rows + 4096


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: tsg.gated_linear(x, x, x, x), lambda: tsg.gated_linear_grad(x, x, x, x, x, x, x, x, x),
                 lambda: tsg.linear_cross_entropy(x, x, None, None, None),
                 lambda: tsg.linear_cross_entropy_grad(None, x, x, None, None, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="act"):
        tsg.gated_linear(x, x, x, x, act="relu")
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        tsg.gated_linear(x.float(), x, x, x)
