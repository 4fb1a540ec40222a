"""The weight gradient's rule for tile and row split: the shapes of the GPU tests
take the kernels that they are there for, and every split has rows."""

import pytest

import persistent_tile_scheduled_amd as tsg
from tests.wgrad_rule import LARGE, LARGE_SPLIT, SMALL, SMALL_SPLIT, wgrad_shape


@pytest.mark.parametrize("shapes,tile,split", [(LARGE, 256, False), (LARGE_SPLIT, 256, True), (SMALL, 128, False),
                                               (SMALL_SPLIT, 128, True)])
def test_the_gpu_tests_shapes_take_the_kernels_they_are_for(shapes, tile, split):
    for rows, out, width in shapes:
        t, _, _, _, splits, per = wgrad_shape(rows, out, width)
        assert t == tile and (splits > 1) == split, (rows, out, width)
        if (shapes is not LARGE) or rows == 2600:
            assert per > 40     # room for every way from fp16 to the split dy and back


@pytest.mark.parametrize("rows", [0, 1, 64, 65, 1000, 4096, 65536, 1 << 30, (1 << 31) - 1])
def test_the_splits_cover_the_rows(rows):
    for out, width in ((8, 32), (64, 64), (512, 512), (1000, 2016), (8192, 64), (4096, 4096), (16384, 16384)):
        tile, mb, nb, slabs, splits, per = wgrad_shape(rows, out, width)
        assert tile in (128, 256) and 1 <= splits <= 256
        assert (mb - 1) * tile < out <= mb * tile and (nb - 1) * tile < width <= nb * tile
        assert slabs == (rows + 63) // 64 and splits * per >= slabs and (splits - 1) * per < max(slabs, 1)
        assert tsg.mx_weight_grad_workspace(rows, out, width) == (4 * splits * out * width if splits > 1 else 0)
