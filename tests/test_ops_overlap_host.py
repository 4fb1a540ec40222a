"""Outputs over inputs are refused: kernels read their inputs while other
workgroups already write (layer_norm_grad of a small matrix reads dy and x a second
time, column by column).  Matrices that only lie between each other's rows do not
overlap.  No GPU: every call here is turned down before anything is launched."""

import ctypes
import os
import subprocess
import tempfile

import pytest

import persistent_tile_scheduled_amd as tsg
from persistent_tile_scheduled_amd import _build

P = 1 << 20          # addresses that nothing reads
B16, F32 = tsg.BF16, tsg.FP32


def at(i):
    return P + (i << 24)


def _norm(x=at(0), ldx=64, g=at(1), b=at(2), y=at(3), ldy=64, mean=at(4), rstd=at(5), codes=None, scales=None, rows=4):
    return tsg.load().tsgemm_layer_norm(rows, 64, B16, B16, x, ldx, g, b, 1e-5, y, ldy, mean, rstd, codes, scales, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(y=at(0)), "y overlaps x"),
    (dict(y=at(0) + 126), "y overlaps x"),
    (dict(y=at(0) + 4 * 128 - 2), "y overlaps x"),
    (dict(y=at(0) - 4 * 128 + 2), "y overlaps x"),
    (dict(ldx=128, ldy=128, y=at(0) + 126), "y overlaps x"),
    (dict(ldx=128, ldy=128, y=at(0) + 2 * 256 + 2), "y overlaps x"),
    (dict(ldx=128, y=at(0) + 128, ldy=72), "y overlaps x"),
    (dict(y=at(1)), "y overlaps gamma"),
    (dict(mean=at(2) + 124), "mean overlaps beta"),
    (dict(rstd=at(0) + 508), "rstd overlaps x"),
    (dict(rstd=at(4) + 12), "rstd overlaps mean"),
    (dict(codes=at(0), scales=at(6)), "codes overlaps x"),
    (dict(codes=at(6), scales=at(0) + 508), "scales overlaps x"),
    (dict(codes=at(6), scales=at(6) + 252), "scales overlaps codes"),
    (dict(codes=at(3), scales=at(6)), "codes overlaps y"),
])
def test_layer_norm_refuses_overlaps(kw, needle):
    assert _norm(**kw) == tsg.EINVAL
    assert needle in tsg.last_error()


@pytest.mark.parametrize("kw,needle", [
    (dict(dx=at(0)), "dx overlaps dy"),
    (dict(dx=at(1)), "dx overlaps x"),
    (dict(dx=at(1) + 64), "dx overlaps x"),
    (dict(dg=at(2)), "dgamma overlaps gamma"),
    (dict(db=at(3)), "dbeta overlaps mean"),
    (dict(db=at(6)), "dbeta overlaps dgamma"),
    (dict(ws=at(0)), "workspace overlaps dy"),
    (dict(ws=at(5)), "workspace overlaps dx"),
])
def test_layer_norm_grad_refuses_overlaps(kw, needle):
    a = dict(dy=at(0), x=at(1), g=at(2), mean=at(3), rstd=at(4), dx=at(5), dg=at(6), db=at(7), ws=at(8))
    a.update(kw)
    rc = tsg.load().tsgemm_layer_norm_grad(4, 64, B16, B16, a["dy"], 64, a["x"], 64, a["g"], a["mean"], a["rstd"], a["dx"], 64,
                                           a["dg"], a["db"], a["ws"], 1 << 20, None)
    assert rc == tsg.EINVAL
    assert needle in tsg.last_error()


def test_conversions_refuse_overlaps():
    lib = tsg.load()
    assert lib.tsgemm_mx_quantize(4, 64, B16, at(0), 64, at(0), at(1), None) == tsg.EINVAL
    assert "codes overlaps x" in tsg.last_error()
    assert lib.tsgemm_mx_quantize(4, 64, B16, at(0), 64, at(1), at(0) + 508, None) == tsg.EINVAL
    assert "scales overlaps x" in tsg.last_error()
    assert lib.tsgemm_mx_dequantize(4, 64, B16, at(0), at(1), at(0) - 510, 64, None) == tsg.EINVAL
    assert "out overlaps codes" in tsg.last_error()
    assert lib.tsgemm_mx_dequantize(4, 64, B16, at(0), at(1), at(1), 64, None) == tsg.EINVAL
    assert "out overlaps scales" in tsg.last_error()


@pytest.mark.parametrize("kw,needle", [
    (dict(dw=at(0)), "dw overlaps dy"),
    (dict(dw=at(1)), "dw overlaps codes"),
    (dict(dw=at(2)), "dw overlaps scales"),
    (dict(ws=at(0)), "workspace overlaps dy"),
    (dict(ws=at(3)), "workspace overlaps dw"),
])
def test_weight_grad_refuses_overlaps(kw, needle):
    a = dict(dy=at(0), codes=at(1), scales=at(2), dw=at(3), ws=at(4))
    a.update(kw)
    need = tsg.mx_weight_grad_workspace(65536, 64, 64)
    assert need > 0
    rc = tsg.load().tsgemm_mx_weight_grad(65536, 64, 64, B16, F32, a["dy"], 64, a["codes"], a["scales"], a["dw"], a["ws"], need, None)
    assert rc == tsg.EINVAL
    assert needle in tsg.last_error()


SHIM = """
#include "tsgemm_overlap.h"
extern "C" int overlap(int64_t p, int64_t rows, int64_t bytes, int64_t pitch, int64_t q, int64_t rows2, int64_t bytes2, int64_t pitch2) {
    const tsg::Region a = {(const void*)p, rows, bytes, pitch}, b = {(const void*)q, rows2, bytes2, pitch2};
    const tsg::Extent e = tsg::extent(a), f = tsg::extent(b);
    const bool shared = tsg::overlap(a, b);
    return shared && !(e.from < f.to && f.from < e.to) ? 2 : shared;      // the extents never say no to one
}
"""


def test_overlap_is_exact():
    """Against the sets of bytes, for all small matrices and distances."""
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "o.so")
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-x", "c++", "-", "-I", _build.CSRC, "-o", out], input=SHIM,
                       text=True, check=True)
        f = ctypes.CDLL(out).overlap
    f.argtypes = [ctypes.c_int64] * 8

    def covered(p, rows, size, pitch):
        return {p + r * pitch + b for r in range(rows) for b in range(size)}

    shapes = [(r, n, n + gap) for r in (0, 1, 2, 3, 5) for n in (1, 2, 3) for gap in (0, 1, 2, 5)]
    sets = {s: covered(0, *s) for s in shapes}
    for s in shapes:
        for t in shapes:
            for q in range(-34, 35):
                want = any(b + q in sets[s] for b in sets[t])
                assert f(1000, *s, 1000 + q, *t) == want, (s, t, q)
    assert not f(0, 4, 4, 4, 0, 4, 4, 4)       # a tensor that is not there
