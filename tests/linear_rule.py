"""What the linear layers' rules say of a shape, from their own source."""

import ctypes
import functools
import os
import subprocess
import tempfile

from persistent_tile_scheduled_amd import _build

_SHIM = """
#include "tsgemm_linear_shape.h"
extern "C" int64_t piece(int64_t rows, int64_t vocab) { return tsg::vocab_piece(rows, vocab); }
extern "C" void shape(int64_t M, int64_t N, int64_t slabs, int halves, int may_split, int64_t* a) {
    const tsg::LinShape s = tsg::linear_shape(M, N, slabs, halves != 0, may_split != 0);
    a[0] = s.tile; a[1] = s.m_blocks; a[2] = s.n_blocks; a[3] = s.splits; a[4] = s.per_split;
}
extern "C" int few(int64_t rows, int64_t columns, int64_t width, int weights) {
    return tsg::takes_few(tsg::linear_shape(rows, columns, (width + 63) / 64, weights == 2, false), rows, columns, width, weights);
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
    lib.few.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int]
    return lib


def vocab_piece(rows, vocab):
    return _lib().piece(rows, vocab)


def linear_shape(M, N, slabs, halves, may_split):
    """tile, m_blocks, n_blocks, splits, slabs per split"""
    a = (ctypes.c_int64 * 5)()
    _lib().shape(M, N, slabs, halves, may_split, a)
    return tuple(a)


def takes_few(rows, columns, width, weights):
    return bool(_lib().few(rows, columns, width, weights))


# weights, rows, width, columns of the GPU tests by the kernel that the rule gives them
FEW = [(1, 1, 512, 50001), (1, 16, 1000, 50001), (1, 17, 264, 50001), (1, 32, 4096, 9001), (2, 1, 1024, 65536), (2, 16, 520, 20001),
       (2, 32, 4096, 4100)]
TILE = [(1, 17, 512, 131072), (1, 32, 1000, 50001), (1, 24, 1000, 130999), (1, 31, 520, 65501), (2, 32, 1024, 65536), (2, 28, 1000, 65529)]
