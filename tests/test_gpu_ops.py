"""Layer norm and its gradient, the MX conversions and the weight gradient from
an MX activation, on the GPU against plain fp64 formulas.

Tolerances (derived, per element).  u = 2^-24 is the fp32 rounding, e the output
type's half step (bf16 2^-8, fp16 2^-11, fp32 2^-24 relative; fp16 also 2^-25
absolute, its subnormals' half step).
  * A sum of n terms taken by one thread's chain, lanes and waves in turn passes
    at most 128 roundings at the widths tested: |error| <= 128 u sum|terms|.
  * layer norm: mean is off by 128 u mean|x|, rstd relatively by 128 u (the
    mean's error enters squared), so y by
      e |y| + 2 * 128 u (|h gamma| + |gamma| rstd mean|x| + |beta|).
  * gradient: dx by e |dx| + 2 * 128 u rstd (|g| + mean|g| + |h| mean|g h|),
    dgamma and dbeta by e |sum| + 128 u sum|terms|.
  * weight gradient: e |dw| + (2 rows + 64) u sum|terms|: the matrix core's and
    the splits' fp32 additions, each at most one unit in the last place off.
Conversions are compared for equality.
"""

import numpy as np
import pytest
import torch

import oracle
import persistent_tile_scheduled_amd as tsg
from workloads import mx_encode

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
FP16, BF16, FP32 = torch.float16, torch.bfloat16, torch.float32


def _half(t):
    return torch.finfo(t).eps / 2


def _rand(rows, width, dtype, seed, scale=1.0, shift=0.25):
    g = torch.Generator().manual_seed(seed)
    spread = torch.exp(0.5 * torch.randn(width, generator=g))
    x = torch.randn((rows, width), generator=g) * spread * torch.exp(0.3 * torch.randn((rows, 1), generator=g)) + shift
    return (x * scale).to(dtype).to(DEV)


def _weights(width, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.1 * torch.randn(width, generator=g)).to(dtype).to(DEV), (0.1 * torch.randn(width, generator=g)).to(dtype).to(DEV))


def _held(rows, width):
    return (torch.full((rows, width), 0x55, dtype=torch.uint8, device=DEV),
            torch.full((rows, width // 32), 0x55, dtype=torch.uint8, device=DEV))


def _norm64(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(dim=1)
    rstd = ((x - mean[:, None]).square().mean(dim=1) + eps).pow(-0.5)
    h = (x - mean[:, None]) * rstd[:, None]
    return h * gamma.double() + beta.double(), mean, rstd, h


def _norm_bound(y, mean, rstd, h, x, gamma, beta, dtype):
    a = (h * gamma.double()).abs() + (gamma.double().abs() * (rstd * x.double().abs().mean(dim=1))[:, None]) + beta.double().abs()
    return _half(dtype) * y.abs() + 256 * U * a + (2.0 ** -25 if dtype == FP16 else 0.0)


def _check(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got - want).abs()
    bad = (err > bound).sum().item()
    assert bad == 0, f"{what}: {bad} of {got.numel()} outside, worst {(err / bound.clamp_min(1e-300)).max().item():.3g} of the bound"


NORM_SHAPES = [(1, 1), (3, 7), (5, 31), (64, 32), (9, 64), (70, 100), (33, 128), (17, 250), (130, 512), (12, 513), (7, 1000),
               (300, 1024), (6, 1025), (19, 2049), (2, 4000), (5, 4096), (3, 8192), (2, 8200), (3, 16384), (2, 16392), (2, 30001),
               (3, 32768), (2, 32776), (2, 40001), (1, 131072)]


@pytest.mark.parametrize("dtype,wdtype", [(FP16, FP16), (FP16, FP32), (BF16, BF16), (BF16, FP32), (FP32, FP32)], ids=str)
def test_layer_norm(dtype, wdtype):
    for rows, width in NORM_SHAPES:
        x = _rand(rows, width, dtype, seed=rows + width)
        gamma, beta = _weights(width, wdtype, seed=width)
        y, mean, rstd, h = _norm64(x, gamma, beta, 1e-5)
        buf = torch.full((rows * width + 64,), 123.0, dtype=dtype, device=DEV)
        got = buf[: rows * width].view(rows, width)
        gm, gr = torch.full((rows + 8,), 7.0, device=DEV), torch.full((rows + 8,), 7.0, device=DEV)
        tsg.layer_norm(x, gamma, beta, 1e-5, y=got, mean=gm[:rows], rstd=gr[:rows])
        torch.cuda.synchronize()
        what = f"{rows}x{width}"
        assert (buf[rows * width:] == 123.0).all() and (gm[rows:] == 7.0).all() and (gr[rows:] == 7.0).all(), what
        _check(got, y, _norm_bound(y, mean, rstd, h, x, gamma, beta, dtype), what)
        _check(gm[:rows], mean, 128 * U * x.double().abs().mean(dim=1) + 1e-30, what + " mean")
        # the two-value subtraction x - mean costs mean|x| u more in the deviation
        _check(gr[:rows], rstd, 256 * U * rstd * (1 + (rstd * x.double().abs().mean(dim=1)).square()), what + " rstd")


def test_layer_norm_without_weights_and_statistics():
    for rows, width in ((5, 96), (4, 3000)):
        x = _rand(rows, width, BF16, 3)
        one, zero = torch.ones(width, device=DEV), torch.zeros(width, device=DEV)
        y = torch.empty_like(x)
        for gamma, beta in ((None, None), (_weights(width, FP32, 1)[0], None), (None, _weights(width, BF16, 1)[1])):
            tsg.layer_norm(x, gamma, beta, 1e-5, y=y)
            g, b = one if gamma is None else gamma, zero if beta is None else beta
            w, mean, rstd, h = _norm64(x, g, b, 1e-5)
            _check(y, w, _norm_bound(w, mean, rstd, h, x, g, b, BF16), f"{rows}x{width}")


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32], ids=str)
def test_layer_norm_to_codes(dtype):
    """The codes of an fp32 layer norm are those of its fp32 values, except
    where fp32 lands on the other side of a rounding: there they are
    neighbours.  y and the codes of one call come from the same values."""
    for rows, width in ((3, 32), (40, 64), (9, 96), (21, 512), (5, 544), (7, 1024), (6, 1056), (11, 4000), (3, 8192), (2, 16384),
                        (2, 20000), (2, 32768), (2, 40000)):
        x = _rand(rows, width, dtype, seed=rows * width)
        gamma, beta = _weights(width, FP32, seed=width)
        codes, scales = _held(rows, width)
        y = torch.empty_like(x)
        mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        tsg.layer_norm(x, gamma, beta, 1e-5, y=y, mean=mean, rstd=rstd, codes=codes, scales=scales)
        only, only_s = _held(rows, width)
        tsg.layer_norm(x, gamma, beta, 1e-5, codes=only, scales=only_s)
        torch.cuda.synchronize()
        assert torch.equal(codes, only) and torch.equal(scales, only_s)
        w, m64, r64, h = _norm64(x, gamma, beta, 1e-5)
        _check(y, w, _norm_bound(w, m64, r64, h, x, gamma, beta, dtype), f"{rows}x{width}")
        value = torch.from_numpy(oracle.e4m3_decode(codes.cpu().numpy()) *
                                 np.repeat(oracle.e8m0_decode(scales.cpu().numpy()), 32, axis=1)).to(DEV)
        top = w.abs().view(rows, -1, 32).amax(dim=2).repeat_interleave(32, dim=1)
        slack = _norm_bound(w, m64, r64, h, x, gamma, beta, FP32)
        # half a step of E4M3: 2^-4 of the value or of E4M3's least normal number
        # at the block's scale, whose 448 ... 512 are held at 448
        step = 2.0 ** -4 * torch.maximum(w.abs(), top * 2.0 ** -14) + torch.where(w.abs() > 0.87 * top, top / 8, torch.zeros_like(top))
        _check(value, w, step * (1 + 2.0 ** -10) + 2 * slack, f"{rows}x{width} codes")
        if dtype == FP32:  # y in fp32 is what was encoded
            c, s = mx_encode(y.cpu().double().numpy())
            assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)


def test_layer_norm_odd_rows_stay_alone():
    """A row with a NaN or an infinity, a constant row, one of the type's lowest
    value and an empty-looking (all zero) row leave the others as they are."""
    for width in (64, 608, 4096, 40000):
        for dtype in (FP16, BF16):
            x = _rand(12, width, dtype, 5)
            gamma, beta = _weights(width, dtype, 6)
            ref, odd = torch.empty_like(x), torch.empty_like(x)
            tsg.layer_norm(x, gamma, beta, 1e-5, y=ref)
            z = x.clone()
            z[1, width // 2] = float("nan")
            z[3, 0] = float("inf")
            z[5] = 0
            z[7] = torch.finfo(dtype).min
            z[9, width - 1] = -float("inf")
            codes, scales = _held(12, width)
            mean, rstd = torch.empty(12, device=DEV), torch.empty(12, device=DEV)
            tsg.layer_norm(z, gamma, beta, 1e-5, y=odd, mean=mean, rstd=rstd, codes=codes, scales=scales)
            keep = [0, 2, 4, 6, 8, 10, 11]
            assert torch.equal(odd[keep], ref[keep])
            for r in (1, 3, 9):
                assert torch.isnan(odd[r].float()).all() and ((codes[r] & 0x7F) == 0x7F).all()
            assert torch.equal(odd[5], beta)
            assert ((codes[keep] & 0x7F) != 0x7F).all()
            assert mean[5] == 0
            if dtype == FP16:   # the constant row: its deviations are the mean's rounding, at most
                assert torch.isfinite(odd[7].float()).all()


def _grad64(dy, x, gamma, mean, rstd):
    n = x.shape[1]
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    dy = dy.double()
    g = dy * gamma.double()
    c1, c2 = g.mean(dim=1, keepdim=True), (g * h).mean(dim=1, keepdim=True)
    r = rstd.double()[:, None]
    dx = (g - c1 - h * c2) * r
    size = r * (g.abs() + g.abs().mean(dim=1, keepdim=True) + h.abs() * (g * h).abs().mean(dim=1, keepdim=True))
    return dx, size, (dy * h).sum(dim=0), (dy * h).abs().sum(dim=0), dy.sum(dim=0), dy.abs().sum(dim=0)


GRAD_SHAPES = [(1, 1), (3, 7), (5, 31), (64, 32), (9, 64), (700, 100), (33, 128), (2000, 250), (3000, 512), (12, 513), (7, 1000),
               (300, 1024), (6, 1025), (19, 2049), (2, 4000), (600, 4096), (530, 8192), (2, 8200), (520, 8256), (3, 16384), (2, 16392),
               (300, 16500), (2, 40001)]


@pytest.mark.parametrize("dtype,wdtype", [(FP16, FP16), (FP16, FP32), (BF16, BF16), (BF16, FP32), (FP32, FP32)], ids=str)
def test_layer_norm_grad(dtype, wdtype):
    for rows, width in GRAD_SHAPES:
        x, dy = _rand(rows, width, dtype, rows + width), _rand(rows, width, dtype, rows * width + 1, scale=0.05, shift=0.0)
        gamma, beta = _weights(width, wdtype, seed=width)
        _, mean, rstd, _ = _norm64(x, gamma, beta, 1e-5)
        mean, rstd = mean.float(), rstd.float()
        buf = torch.full((rows * width + 64,), 123.0, dtype=dtype, device=DEV)
        dx = buf[: rows * width].view(rows, width)
        dg, db = (torch.full((width + 16,), 7.0, dtype=wdtype, device=DEV) for _ in range(2))
        need = tsg.layer_norm_grad_workspace(rows, width)
        ws = torch.full((need // 4 + 16,), float("nan"), device=DEV)
        tsg.layer_norm_grad(dy, x, gamma, mean, rstd, dx, dg[:width], db[:width], workspace=ws[: need // 4])
        torch.cuda.synchronize()
        what = f"{rows}x{width}"
        assert (buf[rows * width:] == 123.0).all() and (dg[width:] == 7.0).all() and (db[width:] == 7.0).all(), what
        assert torch.isnan(ws[need // 4:]).all(), what + ": wrote past the workspace"
        wx, size, wg, mg, wb, mb = _grad64(dy, x, gamma, mean, rstd)
        tiny = 2.0 ** -25 if dtype == FP16 else 1e-40
        wtiny = 2.0 ** -25 if wdtype == FP16 else 1e-40
        _check(dx, wx, _half(dtype) * wx.abs() + 256 * U * size + tiny, what + " dx")
        _check(dg[:width], wg, _half(wdtype) * wg.abs() + 128 * U * mg + wtiny, what + " dgamma")
        _check(db[:width], wb, _half(wdtype) * wb.abs() + 128 * U * mb + wtiny, what + " dbeta")
        # without the sums, with one of them, without gamma: the same dx, the same sum
        one = torch.empty_like(dx)
        tsg.layer_norm_grad(dy, x, gamma, mean, rstd, one)
        assert torch.equal(one, dx), what
        only = torch.empty(width, dtype=wdtype, device=DEV)
        tsg.layer_norm_grad(dy, x, gamma, mean, rstd, one, dbeta=only)
        assert torch.equal(only, db[:width]) and torch.equal(one, dx), what


def test_layer_norm_grad_empty_and_plain():
    dg, db = torch.full((96,), 7.0, device=DEV), torch.full((96,), 7.0, device=DEV)
    x, none = torch.empty((0, 96), dtype=BF16, device=DEV), torch.empty(0, device=DEV)
    tsg.layer_norm_grad(x, x, torch.ones(96, device=DEV), none, none, x, dg, db)
    assert (dg == 0).all() and (db == 0).all()
    x, dy = _rand(40, 96, BF16, 1), _rand(40, 96, BF16, 2, scale=0.05, shift=0.0)
    mean, rstd = torch.empty(40, device=DEV), torch.empty(40, device=DEV)
    tsg.layer_norm(x, None, None, 1e-5, y=torch.empty_like(x), mean=mean, rstd=rstd)
    dx = torch.empty_like(x)
    tsg.layer_norm_grad(dy, x, None, mean, rstd, dx, dg, db)
    wx, size, wg, mg, wb, mb = _grad64(dy, x, torch.ones(96, device=DEV), mean, rstd)
    _check(dx, wx, _half(BF16) * wx.abs() + 256 * U * size, "dx")
    _check(dg, wg, U * wg.abs() + 128 * U * mg, "dgamma")


def test_layer_norm_grad_against_differences():
    """d/dt of sum(dy * layer_norm(x + t p)) by central differences in fp64."""
    rows, width = 6, 200
    x, dy = _rand(rows, width, FP32, 1), _rand(rows, width, FP32, 2, scale=0.1, shift=0.0)
    gamma, beta = _weights(width, FP32, 3)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    tsg.layer_norm(x, gamma, beta, 1e-5, y=torch.empty_like(x), mean=mean, rstd=rstd)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    tsg.layer_norm_grad(dy, x, gamma, mean, rstd, dx, dg, db)

    def f(x, g, b):
        return (dy.double() * _norm64(x, g, b, 1e-5)[0]).sum()

    t = 1e-5
    x, g, b = x.double(), gamma.double(), beta.double()
    for seed, got, args in ((1, dx, lambda p: ((x + t * p, g, b), (x - t * p, g, b))),
                            (2, dg, lambda p: ((x, g + t * p, b), (x, g - t * p, b))),
                            (3, db, lambda p: ((x, g, b + t * p), (x, g, b - t * p)))):
        p = torch.randn(got.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).to(DEV)
        hi, lo = args(p)
        slope = (f(*hi) - f(*lo)) / (2 * t)
        size = (got.double() * p).abs().sum()
        # the difference is off by t^2 of the third derivative, far below 1e-6 of the terms; got by its bound
        assert abs((got.double() * p).sum() - slope) <= 1e-5 * size


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32], ids=str)
def test_mx_quantize_matches_the_definition(dtype):
    g = torch.Generator().manual_seed(11)
    for rows, width in ((1, 32), (3, 64), (7, 96), (33, 4000), (130, 1024)):
        x = torch.randn((rows, width), generator=g) * torch.exp2(torch.randint(-30, 12, (rows, width // 32), generator=g).float()).repeat_interleave(32, 1)
        x[torch.rand((rows, width), generator=g) < 0.1] = 0
        x = x.to(dtype)
        flat = x.view(-1)
        top = torch.finfo(dtype).max
        edges = torch.tensor([448.0, 456.0, 464.0, 480.0, 496.0, 511.0, 512.0, -448.0, 1.0, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, -0.0, 256.0])
        flat[:16] = edges.to(dtype)
        x[-1, -32:] = 0
        if rows > 2:
            x[1, :32] = torch.finfo(dtype).smallest_normal * torch.linspace(0.01, 1, 32).to(dtype)   # subnormals
            x[1, 32:64] = torch.linspace(-1, 1, 32).to(dtype) * top
        buf, scales = _held(rows, width)
        tsg.mx_quantize(x.to(DEV), buf, scales)
        c, s = mx_encode(x.double().numpy())
        assert np.array_equal(scales.cpu().numpy(), s), (rows, width)
        got = buf.cpu().numpy()
        # a zero's code keeps the sign that its value has; the definition's numbers are compared
        assert np.array_equal(oracle.e4m3_decode(got), oracle.e4m3_decode(c)), (rows, width)


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32], ids=str)
def test_mx_quantize_values_that_are_no_numbers(dtype):
    x = _rand(16, 256, dtype, 4)
    base, bs = _held(16, 256)
    tsg.mx_quantize(x, base, bs)
    z = x.clone()
    at = [(1, 5, float("nan")), (2, 40, float("inf")), (3, 255, -float("inf")), (5, 64, float("nan")), (5, 65, float("inf"))]
    for r, c, v in at:
        z[r, c] = v
    z[9, 96:128] = float("nan")
    codes, scales = _held(16, 256)
    tsg.mx_quantize(z, codes, scales)
    want = z.clone()
    for r, c, _ in at:
        want[r, c] = 0                       # the others are held as if it were not there
    want[9, 96:128] = 0
    wc, ws = _held(16, 256)
    tsg.mx_quantize(want, wc, ws)
    odd = ~torch.isfinite(z.float())
    assert ((codes[odd] & 0x7F) == 0x7F).all()
    assert torch.equal(codes[~odd], wc[~odd]) and torch.equal(scales, ws)
    back = torch.empty_like(x)
    tsg.mx_dequantize(codes, scales, back)
    assert torch.isnan(back[odd].float()).all() and torch.isfinite(back[~odd].float()).all()


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32], ids=str)
def test_mx_dequantize_every_code_and_scale(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat_interleave(32).repeat(256).view(256, 8192)
    codes[:, 1::2] = codes.flip(1)[:, 1::2]
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 256).contiguous()
    out = torch.full((256, 8192), 3.0, dtype=dtype, device=DEV)
    tsg.mx_dequantize(codes.to(DEV), scales.to(DEV), out)
    v = oracle.e4m3_decode(codes.numpy()) * np.repeat(oracle.e8m0_decode(scales.numpy()), 32, axis=1)
    want = torch.from_numpy(v).float().to(dtype).float()     # at most 4 bits: only the last step rounds
    got = out.cpu().float()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])


def _mx_values(rows, width, seed, spread=3):
    rng = np.random.default_rng(seed)
    c, s = mx_encode(rng.standard_normal((rows, width)), rng, spread)
    v = oracle.e4m3_decode(c) * np.repeat(oracle.e8m0_decode(s), 32, axis=1)
    return torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), torch.from_numpy(v).to(DEV)


WGRAD_SHAPES = [(1, 8, 32), (1, 64, 64), (5, 72, 96), (63, 128, 128), (64, 256, 256), (65, 264, 288), (128, 136, 160), (129, 512, 512),
                (200, 1000, 544), (257, 2048, 320), (1000, 8, 2048), (3000, 256, 96), (4097, 320, 288), (700, 2304, 2080)]


@pytest.mark.parametrize("dtype,gdtype", [(FP16, FP16), (FP16, FP32), (BF16, BF16), (BF16, FP32)], ids=str)
def test_weight_grad(dtype, gdtype):
    for rows, out, width in WGRAD_SHAPES:
        codes, scales, value = _mx_values(rows, width, rows + out + width)
        dy = _rand(rows, out, dtype, seed=rows * 3 + out, scale=0.05, shift=0.0)
        buf = torch.full((out * width + 64,), 123.0, dtype=gdtype, device=DEV)
        dw = buf[: out * width].view(out, width)
        need = tsg.mx_weight_grad_workspace(rows, out, width)
        ws = torch.full((need // 4 + 16,), float("nan"), device=DEV)
        tsg.mx_weight_grad(dy, codes, scales, dw, workspace=ws[: need // 4])
        torch.cuda.synchronize()
        what = f"{rows}x{out}x{width}"
        assert (buf[out * width:] == 123.0).all(), what
        assert torch.isnan(ws[need // 4:]).all(), what + ": wrote past the workspace"
        d = dy.double().t().contiguous()
        want, mag = d @ value, d.abs() @ value.abs()
        _check(dw, want, _half(gdtype) * want.abs() + (2 * rows + 64) * U * mag + (2.0 ** -25 if gdtype == FP16 else 1e-40), what)
        again = torch.empty_like(dw)
        tsg.mx_weight_grad(dy, codes, scales, again)
        assert torch.equal(again, dw), what + ": two calls differ"


@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_weight_grad_exact_sums(dtype):
    """Small integers times powers of two: every partial sum is exact, so the
    result is too, whatever the order; a code that meets the wrong row, column
    or scale shows."""
    for rows, out, width in ((96, 256, 256), (300, 520, 608), (2000, 128, 64)):
        rng = np.random.default_rng(rows)
        c = rng.choice(np.array([0xC0, 0xB8, 0x00, 0x38, 0x40], np.uint8), size=(rows, width))
        s = rng.integers(125, 130, size=(rows, width // 32)).astype(np.uint8)
        v = oracle.e4m3_decode(c) * np.repeat(oracle.e8m0_decode(s), 32, axis=1)
        dy = torch.from_numpy(rng.integers(-3, 4, size=(rows, out)).astype(np.float64))
        dw = torch.empty((out, width), device=DEV)
        tsg.mx_weight_grad(dy.to(dtype).to(DEV), torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), dw)
        assert torch.equal(dw.cpu().double(), dy.t().contiguous() @ torch.from_numpy(v)), (rows, out, width)


@pytest.mark.parametrize("rows,out,width", [(200, 264, 288), (150, 512, 256)])
def test_weight_grad_fp16_keeps_far_scales(rows, out, width):
    """fp16 dy with scales far outside what fp16 can hold: rows whose block
    scale is 2^-60 or 2^40 next to ordinary ones, each tested where it alone
    counts (the others' dy is zero there)."""
    rng = np.random.default_rng(5)
    c, s = mx_encode(rng.standard_normal((rows, width)))
    s[1::3] = 127 - 60
    s[2::3] = 127 + 40
    v = torch.from_numpy(oracle.e4m3_decode(c) * np.repeat(oracle.e8m0_decode(s), 32, axis=1)).to(DEV)
    g = torch.Generator().manual_seed(1)
    for part in range(3):
        dy = torch.zeros((rows, out))
        dy[part::3] = torch.randn((len(range(part, rows, 3)), out), generator=g)
        dy = dy.to(FP16).to(DEV)
        dw = torch.empty((out, width), device=DEV)
        tsg.mx_weight_grad(dy, torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), dw)
        d = dy.double().t().contiguous()
        want, mag = d @ v, d.abs() @ v.abs()
        _check(dw, want, (2 * rows + 64) * U * mag + U * want.abs(), f"part {part}")


def test_weight_grad_fp16_infinite_dy():
    """An infinite dy makes its row of dw infinite, with the sign of the codes, in
    slabs of ordinary and of far scales alike; the other rows stay."""
    rows, out, width = 130, 72, 96
    codes = torch.full((rows, width), 0x38, dtype=torch.uint8, device=DEV)      # 1
    codes[:, 1::2] = 0xB8                                                        # -1
    dy = _rand(rows, out, FP16, 7, scale=0.05, shift=0.0)
    for field in (127, 127 + 60):
        scales = torch.full((rows, width // 32), field, dtype=torch.uint8, device=DEV)
        base, odd = torch.empty((out, width), device=DEV), torch.empty((out, width), device=DEV)
        tsg.mx_weight_grad(dy, codes, scales, base)
        z = dy.clone()
        z[77, 13] = float("inf")
        tsg.mx_weight_grad(z, codes, scales, odd)
        assert (odd[13, 0::2] == float("inf")).all() and (odd[13, 1::2] == -float("inf")).all(), field
        keep = [i for i in range(out) if i != 13]
        assert torch.equal(odd[keep], base[keep])


def test_weight_grad_empty_and_odd_values():
    dw = torch.full((64, 96), 7.0, device=DEV)
    tsg.mx_weight_grad(torch.empty((0, 64), dtype=BF16, device=DEV), torch.empty((0, 96), dtype=torch.uint8, device=DEV),
                       torch.empty((0, 3), dtype=torch.uint8, device=DEV), dw)
    assert (dw == 0).all()
    for dtype in (FP16, BF16):
        codes, scales, value = _mx_values(100, 320, 3)
        dy = _rand(100, 264, dtype, 4, scale=0.05, shift=0.0)
        base, odd = torch.empty((264, 320), device=DEV), torch.empty((264, 320), device=DEV)
        tsg.mx_weight_grad(dy, codes, scales, base)
        codes[50, 33] = 0x7F          # a NaN code: column 33
        scales[70, 9] = 0xFF          # a NaN scale: columns 288 .. 319
        dy[20, 100] = float("nan")    # row 100
        tsg.mx_weight_grad(dy, codes, scales, odd)
        bad = torch.zeros((264, 320), dtype=torch.bool, device=DEV)
        bad[:, 33] = True
        bad[:, 288:] = True
        bad[100] = True
        assert torch.isnan(odd[bad]).all()
        assert torch.equal(odd[~bad], base[~bad])


@pytest.mark.parametrize("dtype", [FP16, BF16, FP32], ids=str)
def test_row_strides_and_odd_addresses(dtype):
    """Rows apart from each other and beginning at any element: the results are
    those of packed, aligned copies, and what lies between is left alone."""
    for rows, width in ((9, 64), (7, 992), (5, 1056), (3, 8192), (2, 40000)):
        big = _rand(rows, width + 13, dtype, 3)
        bdy = _rand(rows, width + 11, dtype, 4, scale=0.05, shift=0.0)
        x, dy = big[:, 5:5 + width], bdy[:, 1:1 + width]
        gamma, beta = (torch.cat([t.new_zeros(1), t])[1:] for t in _weights(width, FP32, 5))
        outs = []
        for strided in (False, True):
            xs, ds = (x, dy) if strided else (x.contiguous(), dy.contiguous())

            def empty():
                frame = torch.full((rows, width + 9), 123.0, dtype=dtype, device=DEV)
                return frame, (frame[:, 3:3 + width] if strided else torch.empty((rows, width), dtype=dtype, device=DEV))

            (fy, y), (fd, dx), (fo, back) = empty(), empty(), empty()
            mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
            tsg.layer_norm(xs, gamma, beta, 1e-5, y=y, mean=mean, rstd=rstd)
            dg, db = torch.empty(width, device=DEV), torch.empty(width, device=DEV)
            tsg.layer_norm_grad(ds, xs, gamma, mean, rstd, dx, dg, db)
            codes, scales = _held(rows, width)
            tsg.mx_quantize(xs, codes, scales)
            tsg.mx_dequantize(codes, scales, back)
            if strided:
                for f in (fy, fd, fo):
                    assert (f[:, :3] == 123.0).all() and (f[:, 3 + width:] == 123.0).all()
            outs.append([t.clone() for t in (y, mean, rstd, dx, dg, db, codes, scales, back)])
        for a, b in zip(*outs):
            assert torch.equal(a, b), (rows, width)
    if dtype != FP32:
        big = _rand(130, 320, dtype, 6, scale=0.05, shift=0.0)
        codes, scales, _ = _mx_values(130, 96, 7)
        a, b = torch.empty((264, 96), device=DEV), torch.empty((264, 96), device=DEV)
        tsg.mx_weight_grad(big[:, 16:280], codes, scales, a)
        tsg.mx_weight_grad(big[:, 16:280].contiguous(), codes, scales, b)
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """More than 2^32 bytes a matrix: the rows past that mark come out like the
    same rows alone."""
    rows, width = 70000, 32768
    x = torch.empty((rows, width), dtype=FP16, device=DEV)
    x.fill_(0.5)
    tail = _rand(40, width, FP16, 1)
    x[-40:] = tail
    gamma, beta = _weights(width, FP32, 2)
    codes, scales = torch.empty((rows, width), dtype=torch.uint8, device=DEV), torch.empty((rows, width // 32), dtype=torch.uint8, device=DEV)
    tc, ts = _held(40, width)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    tm, tr = torch.empty(40, device=DEV), torch.empty(40, device=DEV)
    y, ty = torch.empty_like(x), torch.empty_like(tail)
    tsg.layer_norm(x, gamma, beta, 1e-5, y=y, mean=mean, rstd=rstd, codes=codes, scales=scales)
    tsg.layer_norm(tail, gamma, beta, 1e-5, y=ty, mean=tm, rstd=tr, codes=tc, scales=ts)
    for a, b in ((y, ty), (mean, tm), (rstd, tr), (codes, tc), (scales, ts)):
        assert torch.equal(a[-40:], b)
    dx, tdx = torch.empty_like(x), torch.empty_like(tail)
    tsg.layer_norm_grad(x, y, gamma, mean, rstd, dx)
    tsg.layer_norm_grad(tail, ty, gamma, tm, tr, tdx)
    assert torch.equal(dx[-40:], tdx)
    tsg.mx_quantize(x, codes, scales)
    tsg.mx_quantize(tail, tc, ts)
    assert torch.equal(codes[-40:], tc) and torch.equal(scales[-40:], ts)
    tsg.mx_dequantize(codes, scales, y)
    tsg.mx_dequantize(tc, ts, ty)
    assert torch.equal(y[-40:], ty)
    del y, dx, codes, scales
    # the weight gradient of the last rows: the others' dy is zero
    dy = x
    dy[:-40] = 0
    c, s, v = _mx_values(rows, 32, 3)
    dw = torch.empty((width, 32), device=DEV)
    tsg.mx_weight_grad(dy, c, s, dw)
    d = tail.double().t().contiguous()
    want, mag = d @ v[-40:], d.abs() @ v[-40:].abs()
    _check(dw, want, U * want.abs() + 200 * U * mag, "weight gradient past 2^32")


def _everything(x, dy, gamma, beta, out, stream=None):
    """One pass through all five into the tensors of `out`."""
    tsg.layer_norm(x, gamma, beta, 1e-5, y=out["y"], mean=out["mean"], rstd=out["rstd"], codes=out["codes"], scales=out["scales"], stream=stream)
    tsg.mx_weight_grad(dy, out["codes"], out["scales"], out["dw"], stream=stream)
    tsg.layer_norm_grad(out["y"], x, gamma, out["mean"], out["rstd"], out["dx"], out["dg"], out["db"], stream=stream)
    tsg.mx_quantize(out["dx"], out["qc"], out["qs"], stream=stream)
    tsg.mx_dequantize(out["qc"], out["qs"], out["back"], stream=stream)


def _outs(rows, width, n, dtype):
    e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device=DEV)  # noqa: E731
    u8 = torch.uint8
    return {"y": e(rows, width, t=dtype), "mean": e(rows), "rstd": e(rows), "codes": e(rows, width, t=u8), "scales": e(rows, width // 32, t=u8),
            "dw": e(n, width), "dx": e(rows, width, t=dtype), "dg": e(width), "db": e(width), "qc": e(rows, width, t=u8),
            "qs": e(rows, width // 32, t=u8), "back": e(rows, width, t=dtype)}


def test_other_streams():
    rows, width, n = 700, 1056, 136
    gamma, beta = _weights(width, FP32, 1)
    ins = [(_rand(rows, width, BF16, s), _rand(rows, n, BF16, s + 9, scale=0.05, shift=0.0)) for s in (1, 2)]
    alone = [_outs(rows, width, n, BF16) for _ in ins]
    for (x, dy), o in zip(ins, alone):
        _everything(x, dy, gamma, beta, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        both = [_outs(rows, width, n, BF16) for _ in ins]
        torch.cuda.synchronize()
        for s, (x, dy), o in zip(streams, ins, both):
            _everything(x, dy, gamma, beta, o, stream=s)
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            for k in a:
                assert torch.equal(a[k], b[k]), k


def test_graph_replays_match_eager():
    rows, width, n = 520, 544, 264
    gamma, beta = _weights(width, FP32, 1)
    x, dy = _rand(rows, width, FP16, 1), _rand(rows, n, FP16, 2, scale=0.05, shift=0.0)
    o, ref = _outs(rows, width, n, FP16), _outs(rows, width, n, FP16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _everything(x, dy, gamma, beta, o)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _everything(x, dy, gamma, beta, o)
    for seed in (3, 4, 5):
        x.copy_(_rand(rows, width, FP16, seed))
        dy.copy_(_rand(rows, n, FP16, seed + 20, scale=0.05, shift=0.0))
        for t in o.values():
            t.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _everything(x, dy, gamma, beta, ref)
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k], ref[k]), (seed, k)


def test_mx_norm_linear_step():
    """The layer of mx_linear: its outputs and gradients against fp64 on the
    values that its codes stand for."""
    from persistent_tile_scheduled_amd.mx_linear import MxNormLinear
    rows, width, out = 300, 256, 320
    layer = MxNormLinear(width, out, seed=3)
    layer.gamma.copy_(_weights(width, FP32, 4)[0])
    x, dy = _rand(rows, width, BF16, 5), _rand(rows, out, BF16, 6, scale=0.05, shift=0.0)
    y, saved = layer.forward(x)
    dx, grads = layer.backward(dy, saved)
    _, mean, rstd, codes, scales, wcodes, wscales = saved

    def value(c, s):
        return torch.from_numpy(oracle.e4m3_decode(c.view(torch.uint8).cpu().numpy()) *
                                np.repeat(oracle.e8m0_decode(s.view(torch.uint8).cpu().numpy()), 32, axis=1)).to(DEV)

    a, w = value(codes, scales), value(wcodes, wscales)
    want, mag = a @ w.t().contiguous(), a.abs() @ w.abs().t().contiguous()
    _check(y, want, 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag, "y")
    d = dy.double().t().contiguous()
    want, mag = d @ a, d.abs() @ a.abs()
    _check(grads["weight"], want, U * want.abs() + (2 * rows + 64) * U * mag, "weight")
    dn = (dy.double() @ w).to(BF16)
    wx, size, wg, mg, wb, mb = _grad64(dn, x, layer.gamma, mean, rstd)
    # dn is rounded to bf16 from an fp32 sum that may fall on the other side: one step, 2^-7, more
    slack = 2.0 ** -7
    _check(dx, wx, _half(BF16) * wx.abs() + (256 * U + slack) * size, "dx")
    _check(grads["gamma"], wg, (128 * U + slack) * mg, "gamma")
    _check(grads["beta"], wb, (128 * U + slack) * mb, "beta")


SMALL_SHAPES = [(1, 8), (2, 9), (1024, 1024), (1025, 1024), (1024, 1025), (1024, 5), (255, 4096), (100, 4097), (65, 63), (1000, 777)]


@pytest.mark.parametrize("dtype,wdtype", [(FP16, FP16), (BF16, FP32), (FP32, FP32)], ids=str)
def test_layer_norm_grad_about_its_borders(dtype, wdtype):
    """Shapes on both sides of the border between one launch and two, in both
    ways of calling (torch's workspace and stream, and the caller's): the same
    bits, within the bound of test_layer_norm_grad."""
    for rows, width in SMALL_SHAPES:
        x, dy = _rand(rows, width, dtype, rows + 2 * width), _rand(rows, width, dtype, rows * width + 3, scale=0.05, shift=0.0)
        gamma, beta = _weights(width, wdtype, seed=width)
        _, mean, rstd, _ = _norm64(x, gamma, beta, 1e-5)
        mean, rstd = mean.float(), rstd.float()
        outs = []
        for kw in ({}, {"workspace": torch.full((tsg.layer_norm_grad_workspace(rows, width),), 0xFF, dtype=torch.uint8, device=DEV)},
                   {"stream": torch.cuda.current_stream()}):
            dx = torch.full_like(x, 7.0)
            dg, db = (torch.full((width + 16,), 7.0, dtype=wdtype, device=DEV) for _ in range(2))
            tsg.layer_norm_grad(dy, x, gamma, mean, rstd, dx, dg[:width], db[:width], **kw)
            outs.append((dx, dg, db))
            assert (dg[width:] == 7.0).all() and (db[width:] == 7.0).all()
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
        dx, dg, db = outs[0]
        wx, size, wg, mg, wb, mb = _grad64(dy, x, gamma, mean, rstd)
        tiny, wtiny = (2.0 ** -25 if t == FP16 else 1e-40 for t in (dtype, wdtype))
        what = f"{rows}x{width}"
        _check(dx, wx, _half(dtype) * wx.abs() + 256 * U * size + tiny, what + " dx")
        _check(dg[:width], wg, _half(wdtype) * wg.abs() + 128 * U * mg + wtiny, what + " dgamma")
        _check(db[:width], wb, _half(wdtype) * wb.abs() + 128 * U * mb + wtiny, what + " dbeta")


def test_both_ways_of_calling_agree():
    """The extension module (torch's current stream) and the Python marshalling
    (a stream given) make the same calls."""
    rows, width, n = 70, 96, 136
    gamma, beta = _weights(width, BF16, 1)
    x, dy = _rand(rows, width, BF16, 2), _rand(rows, n, BF16, 3, scale=0.05, shift=0.0)
    a, b = _outs(rows, width, n, BF16), _outs(rows, width, n, BF16)
    for o in (a, b):
        o["dg"], o["db"] = o["dg"].bfloat16(), o["db"].bfloat16()
    _everything(x, dy, gamma, beta, a)
    _everything(x, dy, gamma, beta, b, stream=torch.cuda.current_stream())
    for k in a:
        assert torch.equal(a[k], b[k]), k
    with torch.cuda.stream(torch.cuda.Stream()):
        c = _outs(rows, width, n, BF16)
        c["dg"], c["db"] = c["dg"].bfloat16(), c["db"].bfloat16()
        torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
        _everything(x, dy, gamma, beta, c)
        torch.cuda.current_stream().synchronize()
    for k in a:
        assert torch.equal(a[k], c[k]), k


def test_bad_tensors_are_named():
    x, v = _rand(4, 64, BF16, 1), torch.ones(64, device=DEV)
    codes, scales = _held(4, 64)
    with pytest.raises(ValueError, match="gamma"):
        tsg.layer_norm(x, v[:32], v, 1e-5, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="y must be"):
        tsg.layer_norm(x, v, v, 1e-5, y=torch.empty((4, 63), dtype=BF16, device=DEV))
    with pytest.raises(ValueError, match="beta"):
        tsg.layer_norm(x, v, v.bfloat16(), 1e-5, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="contiguous rows"):
        tsg.mx_quantize(x.t(), codes, scales)
    with pytest.raises(ValueError, match="scales"):
        tsg.mx_quantize(x, codes, scales[:, :1])
    with pytest.raises(ValueError, match="codes"):
        tsg.mx_dequantize(codes.bool(), scales, x)
    with pytest.raises(ValueError, match="divisible by 32"):
        tsg.mx_quantize(x[:, :40], codes, scales)
    with pytest.raises(ValueError, match="dw"):
        tsg.mx_weight_grad(x, codes, scales, torch.empty((63, 64), device=DEV))
    with pytest.raises(tsg.TsgemmError, match="no output"):
        tsg.layer_norm(x, v, v, 1e-5)
    with pytest.raises(tsg.TsgemmError, match="divisible by 8"):
        tsg.mx_weight_grad(_rand(4, 60, BF16, 1), codes, scales, torch.empty((60, 64), device=DEV))
