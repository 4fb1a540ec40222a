"""The weight gradient's kernels one by one, on the GPU: both tiles, with and
without a row split, and fp16's ways between its two forms of multiplying.

Tolerance where sums are not exact (derived, per element): e |dw| + (2 rows + 64)
2^-24 sum|terms|, e the output type's half step, 2^-25 more in fp16 (its
subnormals' half step); the matrix core's and the splits' fp32 additions are each
at most one unit in the last place off.  Exact sums are compared for equality."""

import numpy as np
import pytest
import torch

import oracle
import persistent_tile_scheduled_amd as tsg
from tests.wgrad_rule import LARGE, LARGE_SPLIT, SMALL, SMALL_SPLIT, wgrad_shape

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
FP16, BF16, FP32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [(FP16, FP16), (FP16, FP32), (BF16, BF16), (BF16, FP32)]


def _elements():
    return torch.from_numpy(oracle.e4m3_decode(np.arange(256, dtype=np.uint8))).to(DEV)


def _values(codes, scales):
    return _elements()[codes.long()] * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _random(rows, out, width, dtype, seed):
    g = _generator(seed)
    codes = torch.randint(0, 0x7F, (rows, width), generator=g, device=DEV, dtype=torch.uint8)
    codes += (torch.rand((rows, width), generator=g, device=DEV) < 0.5).to(torch.uint8) * 0x80
    scales = torch.randint(117, 124, (rows, width // 32), generator=g, device=DEV, dtype=torch.uint8)
    dy = (0.05 * torch.randn((rows, out), generator=g, device=DEV)).to(dtype)
    return dy, codes, scales


def _whole(rows, out, width, seed):
    """dy of -3 ... 3 and values of -2 ... 2 times 2^-2 ... 2^1: every partial sum is exact."""
    g = _generator(seed)
    pick = torch.tensor([0xC0, 0xB8, 0x00, 0x38, 0x40], dtype=torch.uint8, device=DEV)
    codes = pick[torch.randint(0, 5, (rows, width), generator=g, device=DEV)]
    scales = torch.randint(125, 129, (rows, width // 32), generator=g, device=DEV, dtype=torch.uint8)
    dy = torch.randint(-3, 4, (rows, out), generator=g, device=DEV).double()
    return dy, codes, scales


def _product(dy, value):
    return dy.double().t().contiguous() @ value


@pytest.mark.parametrize("dtype,gdtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,out,width", LARGE + LARGE_SPLIT + SMALL + SMALL_SPLIT)
def test_tiles_and_splits(rows, out, width, dtype, gdtype):
    dy, codes, scales = _random(rows, out, width, dtype, rows + out + width)
    buf = torch.full((out * width + 64,), 123.0, dtype=gdtype, device=DEV)
    dw = buf[: out * width].view(out, width)
    need = tsg.mx_weight_grad_workspace(rows, out, width)
    ws = torch.full((need // 4 + 16,), float("nan"), device=DEV)
    tsg.mx_weight_grad(dy, codes, scales, dw, workspace=ws[: need // 4])
    torch.cuda.synchronize()
    assert (buf[out * width:] == 123.0).all()
    assert torch.isnan(ws[need // 4:]).all(), "wrote past the workspace"
    value = _values(codes, scales)
    want, size = _product(dy, value), _product(dy.abs(), value.abs())
    bound = torch.finfo(gdtype).eps / 2 * want.abs() + (2 * rows + 64) * U * size + (2.0 ** -25 if gdtype == FP16 else 1e-40)
    off = (dw.double() - want).abs()
    assert torch.isfinite(dw).all() and (off <= bound).all(), (off / bound).max().item()
    again = torch.empty_like(dw)
    tsg.mx_weight_grad(dy, codes, scales, again)
    assert torch.equal(again, dw), "two calls differ"


@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
@pytest.mark.parametrize("rows,out,width", LARGE + LARGE_SPLIT + SMALL + SMALL_SPLIT)
def test_exact_sums(rows, out, width, dtype):
    dy, codes, scales = _whole(rows, out, width, rows)
    dw = torch.full((out, width), 7.0, device=DEV)
    tsg.mx_weight_grad(dy.to(dtype), codes, scales, dw)
    assert torch.equal(dw.double(), _product(dy, _values(codes, scales)))


# slabs with a block whose scale is past what fp16 holds
FAR = [(0,), (1,), (2,), (3,), (10,), (11,), (-1,), (-2,), (0, 1), (5, 20), (5, 21), (5, 22), (6, 21), (6, 22), (6, 23), (2, 19, 36),
       (0, 16, 32), (1, 18, 35), (7, -1), tuple(range(3, 40, 2))]


@pytest.mark.parametrize("rows,out,width", [LARGE[-1]] + LARGE_SPLIT[1:] + SMALL + SMALL_SPLIT)
def test_fp16_far_blocks_here_and_there(rows, out, width):
    """One far block in some slabs of every split, ordinary ones elsewhere and dy
    nowhere empty: each slab counts once, whichever form it is multiplied in."""
    _, _, _, slabs, splits, per = wgrad_shape(rows, out, width)
    dy, codes, scales = _whole(rows, out, width, 1)
    d16, near = dy.half(), _product(dy, _values(codes, scales))
    rng = np.random.default_rng(2)
    for far in FAR:
        s, change = scales.clone(), []
        for split in range(splits):
            first, count = split * per, min(per, slabs - split * per)
            for f in far:
                if -count <= f < count:
                    row = min(64 * (first + f % count) + int(rng.integers(0, 64)), rows - 1)
                    change.append((row, int(rng.integers(0, width // 32))))
        change = sorted(set(change))
        at = torch.tensor(change, device=DEV)
        s[at[:, 0], at[:, 1]] = 130                     # 2^3; fp16's last is 2^1
        rest = near.clone()
        for row, block in change:                       # a changed block adds to 32 columns
            c = slice(32 * block, 32 * block + 32)
            v = _elements()[codes[row, c].long()] * (2.0 ** 3 - 2.0 ** (int(scales[row, block]) - 127))
            rest[:, c] += dy[row][:, None] * v[None, :]
        dw = torch.empty((out, width), device=DEV)
        tsg.mx_weight_grad(d16, codes, s, dw)
        assert torch.equal(dw.double(), rest), far


@pytest.mark.parametrize("rows,out,width", [LARGE[1], SMALL_SPLIT[0]])
def test_fp16_far_scales_and_infinities(rows, out, width):
    """Scales of 2^-60 and 2^40, and an infinite dy in an ordinary and in a far slab."""
    dy, codes, scales = _random(rows, out, width, FP16, 3)
    for field in (127 - 60, 127 + 40):
        far = scales.clone()
        far[200:210] = field
        d = dy.clone()
        d[:200] = 0
        d[210:] = 0                                      # the far rows alone count
        dw = torch.empty((out, width), device=DEV)
        tsg.mx_weight_grad(d, codes, far, dw)
        value = _values(codes, far)
        want, size = _product(d, value), _product(d.abs(), value.abs())
        assert ((dw.double() - want).abs() <= U * want.abs() + (2 * rows + 64) * U * size).all(), field
    ones = torch.full_like(codes, 0x38)
    ones[:, 1::2] = 0xB8
    base, odd = torch.empty((out, width), device=DEV), torch.empty((out, width), device=DEV)
    for row, far in ((100, False), (205, True), (rows - 1, False)):
        s = torch.full_like(scales, 127)
        if far:
            s[200:210] = 127 + 60
        tsg.mx_weight_grad(dy, ones, s, base)
        z = dy.clone()
        z[row, out - 3] = float("inf")
        tsg.mx_weight_grad(z, ones, s, odd)
        assert (odd[out - 3, 0::2] == float("inf")).all() and (odd[out - 3, 1::2] == -float("inf")).all()
        odd[out - 3] = base[out - 3]
        assert torch.equal(odd, base)


@pytest.mark.parametrize("rows,out,width", [LARGE[1], LARGE_SPLIT[1]])
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_values_that_are_no_numbers_stay_in_their_places(rows, out, width, dtype):
    dy, codes, scales = _random(rows, out, width, dtype, 4)
    base, odd = torch.empty((out, width), device=DEV), torch.empty((out, width), device=DEV)
    tsg.mx_weight_grad(dy, codes, scales, base)
    codes[501, 33] = 0x7F                    # column 33
    scales[rows - 1, width // 32 - 1] = 0xFF  # the last 32 columns
    dy[20, 301] = float("nan")               # row 301
    tsg.mx_weight_grad(dy, codes, scales, odd)
    bad = torch.zeros((out, width), dtype=torch.bool, device=DEV)
    bad[:, 33] = True
    bad[:, width - 32:] = True
    bad[301] = True
    assert torch.isnan(odd[bad]).all()
    assert torch.equal(odd[~bad], base[~bad])


@pytest.mark.parametrize("fields", [(106, 128), (105, 129), (98, 114)], ids=str)
def test_fp16_every_code_about_the_borders(fields):
    """Every finite code at scales on both sides of the direct form's borders
    (2^-21 and 2^1), where decoded codes are fp16's subnormals or near its top:
    one term an element, whose 11 + 4 bits fp32 holds."""
    low, high = fields
    span = list(range(low, high + 1))
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1)   # [256][256]
    codes[:, 0x7F] = 0
    codes[:, 0xFF] = 0
    g = _generator(5)
    for start in range(0, len(span), 8):                                       # 8 blocks a row
        part = (span * 2)[start:start + 8]
        scales = torch.tensor(part, dtype=torch.uint8, device=DEV).repeat(256, 1)
        scales = torch.stack([scales[r].roll(r) for r in range(256)])
        d = torch.zeros((256, 256), dtype=FP16, device=DEV)
        own = (1 + torch.rand(256, generator=g, device=DEV)).half() * torch.exp2(torch.randint(-8, 8, (256,), generator=g, device=DEV).float()).half()
        d[torch.arange(256), torch.arange(256)] = own                          # row r alone reaches dw's row r
        dw = torch.empty((256, 256), device=DEV)
        tsg.mx_weight_grad(d, codes, scales, dw)
        assert torch.equal(dw.double(), own.double()[:, None] * _values(codes, scales)), part


@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_the_ends_of_the_range(dtype):
    """Scale codes 0 ... 2, where code * scale is rounded to bf16's subnormals, 3,
    from which it is exact, and the top, where it ends with fp32; fp16's sums end
    at 2^122.  One term an element, rows of one scale each alone."""
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(64, 1)
    codes[:, 0x7F] = 0
    codes[:, 0xFF] = 0
    element = _elements()[codes[0].long()]
    for field in (0, 1, 2, 3, 4, 30, 230, 245, 246, 250):
        value = element * 2.0 ** (field - 127)
        held = value.float().bfloat16().double()
        assert torch.equal(held, value) or field < 3 or field > 246
        for power in (-10, 0, 10):
            d = torch.zeros((64, 8), dtype=dtype, device=DEV)
            d[5, 3] = 2.0 ** power
            dw = torch.empty((8, 256), device=DEV)
            tsg.mx_weight_grad(d, codes, torch.full((64, 8), field, dtype=torch.uint8, device=DEV), dw)
            want = held * 2.0 ** power
            end = 2.0 ** (122 if dtype == FP16 else 128)
            want = torch.where(want.abs() >= end, torch.sign(want) * float("inf"), want)
            value_ends = held.abs() >= 2.0 ** 128          # times the other rows' zeros: no number
            assert torch.equal(dw[3].double()[~value_ends], want[~value_ends]), (field, power)
            assert torch.isnan(dw[3][value_ends]).all()
