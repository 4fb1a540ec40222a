"""The rules that choose pieces of the vocabulary and splits of the sum for the gradient of
the linear head's cross entropy, and the kernel for few rows, from their own source, and
the workspaces that follow."""

import pytest

import persistent_tile_scheduled_amd as tsg
from tests.linear_rule import FEW, TILE, linear_shape, takes_few, vocab_piece

MIB = 1 << 20


@pytest.mark.parametrize("rows", [1, 7, 512, 4000, 8192, 16383, 16385, 40000, 100000, 1 << 26])
def test_a_piece_of_the_vocabulary_takes_128_mib(rows):
    """... or 2048 columns where those take more; whole tiles that cover the vocabulary, of one size."""
    for vocab in (1, 255, 257, 2100, 5003, 50001, 131072, 1 << 22, (1 << 22) + 1, 1 << 27):
        p = vocab_piece(rows, vocab)
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
    for M in (1, 33, 300, 512, 2000, 8192, 50000):
        for N in (8, 264, 1000, 2504, 8192):
            for slabs in (1, 2, 9, 64, 189, 2048):
                tile, mb, nb, splits, per = linear_shape(M, N, slabs, False, True)
                assert (mb - 1) * tile < M <= mb * tile and (nb - 1) * tile < N <= nb * tile
                assert (splits - 1) * per < slabs <= splits * per  # every split has slabs
                assert splits == 1 or mb * nb * splits <= (512 if tile == 256 else 1024)


@pytest.mark.parametrize("weights", [1, 2])
def test_the_kernel_for_few_rows(weights):
    """Never above 32 rows, always for one token; of more rows and wider products no more of them."""
    for width in (8, 512, 4096, 8192):
        for columns in (1, 1000, 8192, 50001, 131072):
            takes = [takes_few(rows, columns, width, weights) for rows in range(1, 40)]
            assert takes[0] and not any(takes[32:])
            assert takes == sorted(takes, reverse=True), (width, columns)


@pytest.mark.parametrize("shapes,few", [(FEW, True), (TILE, False)])
def test_the_gpu_tests_shapes_take_the_kernels_they_are_for(shapes, few):
    for weights, rows, width, columns in shapes:
        assert takes_few(rows, columns, width, weights) == few, (weights, rows, width, columns)


@pytest.mark.parametrize("rows", [16, 32])
def test_the_workspace_is_that_of_either_kernel(rows):
    """Parts of 8 bytes a row: 512 workgroups', or two a tile of 256 or 128 columns."""
    for vocab, width in ((5003, 4096), (131072, 512), (200000, 4096)):
        few = takes_few(rows, vocab, width, 1)
        tile, _, nb, _, _ = linear_shape(rows, vocab, -(-width // 64), False, False)
        parts = min(512, -(-vocab // 16)) if few else 2 * nb
        up = lambda n: -(-n // 256) * 256  # noqa: E731
        assert tsg.linear_cross_entropy_workspace(rows, vocab, width) == up(8 * parts * rows) + up(4 * rows)
