"""The rules that choose pieces of the vocabulary and splits of the sum for the gradient of
the linear head's cross entropy, from their own source, and the workspaces that follow."""

import ctypes
import functools
import os
import subprocess
import tempfile

import pytest

import persistent_tile_scheduled_amd as tsg
from persistent_tile_scheduled_amd import _build

_SHIM = """
#include "tsgemm_linear_shape.h"
extern "C" int64_t piece(int64_t rows, int64_t vocab) { return tsg::vocab_piece(rows, vocab); }
extern "C" void shape(int64_t M, int64_t N, int64_t slabs, int halves, int may_split, int64_t* a) {
    const tsg::LinShape s = tsg::linear_shape(M, N, slabs, halves != 0, may_split != 0);
    a[0] = s.tile; a[1] = s.m_blocks; a[2] = s.n_blocks; a[3] = s.splits; a[4] = s.per_split;
}
"""


@functools.cache
def _lib():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "rule.so")
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-x", "c++", "-", "-I", _build.CSRC, "-o", out],
                       input=_SHIM, text=True, check=True)
        lib = ctypes.CDLL(out)
    lib.piece.argtypes, lib.piece.restype = [ctypes.c_int64] * 2, ctypes.c_int64
    lib.shape.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2 + [ctypes.POINTER(ctypes.c_int64)]
    return lib


MIB = 1 << 20


@pytest.mark.parametrize("rows", [1, 7, 512, 4000, 8192, 16383, 16385, 40000, 100000, 1 << 26])
def test_a_piece_of_the_vocabulary_takes_128_mib(rows):
    """... or 2048 columns where those take more; whole tiles that cover the vocabulary, of one size."""
    for vocab in (1, 255, 257, 2100, 5003, 50001, 131072, 1 << 22, (1 << 22) + 1, 1 << 27):
        p = _lib().piece(rows, vocab)
        assert p % 256 == 0 and 2 * rows * p <= max(128 * MIB, 4096 * rows, 512 * rows)
        pieces = -(-vocab // p)
        assert p <= 1 << 22 and (pieces == 1 or p - (vocab - (pieces - 1) * p) < 256 * pieces)
        if 2 * rows * (-(-vocab // 256) * 256) <= 128 * MIB and vocab <= 1 << 22:
            assert pieces == 1


@pytest.mark.parametrize("rows,vocab,width", [(8192, 131072, 4096), (4096, 1 << 20, 512), (100000, 200000, 64), (3, 1 << 27, 64),
                                              (2000, 1 << 18, 8192)])
def test_the_gradients_workspace_is_far_below_the_logits_gradient(rows, vocab, width):
    """A piece of it, the copy of x, and fp32 sums: dx's once if there are several pieces, and those of split
    products, at most 2 x 256 tiles of 256 x 256 (or 2 x 512 of 128 x 128): 2^25 values."""
    held, sums = max(128 * MIB, 4096 * rows), 4 << 25
    bound = held + 2 * rows * width + max(4 * rows * width, sums) + sums + 32 * rows + 8192
    assert tsg.linear_cross_entropy_grad_workspace(rows, vocab, width) <= bound
    assert bound < 2 * rows * vocab


def test_splits_are_as_few_as_that():
    a = (ctypes.c_int64 * 5)()
    for M in (1, 33, 300, 512, 2000, 8192, 50000):
        for N in (8, 264, 1000, 2504, 8192):
            for slabs in (1, 2, 9, 64, 189, 2048):
                _lib().shape(M, N, slabs, 0, 1, a)
                tile, mb, nb, splits, per = a
                assert (mb - 1) * tile < M <= mb * tile and (nb - 1) * tile < N <= nb * tile
                assert (splits - 1) * per < slabs <= splits * per  # every split has slabs
                assert splits == 1 or mb * nb * splits <= (512 if tile == 256 else 1024)
