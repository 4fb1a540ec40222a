"""Which tile and row split the library takes for a weight gradient's shape, from
the rule's own source."""

import ctypes
import functools
import os
import subprocess
import tempfile

from persistent_tile_scheduled_amd import _build

_SHIM = """
#include "tsgemm_wgrad_shape.h"
extern "C" void shape(int64_t rows, int64_t out, int64_t width, int64_t* a) {
    const tsg::WgradShape w = tsg::wgrad_shape(rows, out, width);
    a[0] = w.tile; a[1] = w.m_blocks; a[2] = w.n_blocks; a[3] = w.slabs; a[4] = w.splits; a[5] = w.per_split;
}
"""


@functools.cache
def _lib():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "rule.so")
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-x", "c++", "-", "-I", _build.CSRC, "-o", out],
                       input=_SHIM, text=True, check=True)
        return ctypes.CDLL(out)


def wgrad_shape(rows, out, width):
    """tile, m_blocks, n_blocks, slabs, splits, slabs per split"""
    a = (ctypes.c_int64 * 6)()
    _lib().shape(ctypes.c_int64(rows), ctypes.c_int64(out), ctypes.c_int64(width), a)
    return tuple(a)


# rows, out, width of the GPU tests by the kernel that the rule gives them
LARGE = [(1024, 4096, 4096), (1000, 4104, 4128), (1, 3848, 4064), (65, 4096, 4096), (150, 3848, 4064), (2600, 4104, 4128)]
LARGE_SPLIT = [(32768, 2048, 2048), (20000, 2056, 2080)]
SMALL = [(3000, 2048, 4096)]
SMALL_SPLIT = [(9000, 1288, 1312)]
