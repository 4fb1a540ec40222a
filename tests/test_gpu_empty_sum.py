"""A product without a sum (K = 0) over more values than one launch may have threads for."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg

pytestmark = pytest.mark.gpu


def test_all_of_c_is_zero():
    """C of 2^35 + 2^23 values (64 GiB), 8 of them a thread."""
    dev, M, N = torch.device("cuda:0"), 1 << 20, (1 << 15) + 8
    A, B = torch.empty((M, 0), dtype=torch.float16, device=dev), torch.empty((0, N), dtype=torch.float16, device=dev)
    C = torch.full((M, N), 1.0, dtype=torch.float16, device=dev)
    tsg.Plan(M, N, 0, "fp16", 256, 256, 64, 8, 2).run(A, B, C)
    for i in range(0, M, 1 << 16):
        assert not C[i: i + (1 << 16)].any(), i
    del C
    torch.cuda.empty_cache()
