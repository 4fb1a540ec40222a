"""Refusals and workspace arithmetic of the row operators and the weight
gradient, without a GPU: every bad call is turned down by the C entry before
anything is launched (pointers here are numbers that nothing reads)."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg

P = 1 << 20          # an aligned, never dereferenced address
F16, B16, F32 = tsg.FP16, tsg.BF16, tsg.FP32


def _norm(rows=4, width=64, dt=B16, wdt=B16, x=P, ldx=64, g=P, b=P, eps=1e-5, y=P, ldy=64, mean=P, rstd=P, codes=None,
          scales=None):
    return tsg.load().tsgemm_layer_norm(rows, width, dt, wdt, x, ldx, g, b, eps, y, ldy, mean, rstd, codes, scales, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(rows=-1), ">= 0"),
    (dict(rows=1 << 31), "below 2^31"),
    (dict(width=0), "at least 1"),
    (dict(dt=3, wdt=3), "dtype"),
    (dict(dt=B16, wdt=F16), "weights"),
    (dict(x=None), "x is NULL"),
    (dict(x=P + 1), "aligned"),
    (dict(ldx=63), "row stride of x"),
    (dict(ldy=63), "row stride of y"),
    (dict(y=None), "no output"),
    (dict(y=P + 1), "aligned"),
    (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"),
    (dict(mean=None), "together"),
    (dict(mean=P + 2), "aligned"),
    (dict(g=P + 1), "aligned"),
    (dict(codes=P), "codes or scales"),
    (dict(scales=P), "codes or scales"),
    (dict(codes=P + 8, scales=P), "16-byte"),
    (dict(codes=P, scales=P + 2), "4-byte"),
    (dict(width=40, codes=P, scales=P), "divisible by 32"),
])
def test_layer_norm_refuses(kw, needle):
    assert _norm(**kw) == tsg.EINVAL
    assert needle in tsg.last_error()


def _grad(rows=4, width=64, dt=B16, wdt=F32, dy=P, lddy=64, x=P, ldx=64, g=P, mean=P, rstd=P, dx=P, lddx=64, dg=P, db=P,
          ws=P, size=1 << 30):
    return tsg.load().tsgemm_layer_norm_grad(rows, width, dt, wdt, dy, lddy, x, ldx, g, mean, rstd, dx, lddx, dg, db, ws,
                                             size, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(rows=-1), ">= 0"),
    (dict(width=0), "at least 1"),
    (dict(dt=0), "dtype"),
    (dict(wdt=F16), "weights"),
    (dict(dy=None), "dy is NULL"),
    (dict(x=P + 1), "aligned"),
    (dict(dx=None), "dx is NULL"),
    (dict(lddx=10), "row stride of dx"),
    (dict(mean=None), "mean and rstd"),
    (dict(rstd=P + 1), "mean and rstd"),
    (dict(dg=P + 2), "aligned"),
    (dict(ws=None), "workspace"),
    (dict(ws=P + 8), "workspace"),
    (dict(size=8), "workspace"),
])
def test_layer_norm_grad_refuses(kw, needle):
    assert _grad(**kw) == tsg.EINVAL
    assert needle in tsg.last_error()


def test_layer_norm_grad_workspace():
    assert tsg.layer_norm_grad_workspace(0, 64) == 0
    for rows, width in ((1, 1), (7, 1000), (8192, 8192), (3, 100000)):
        n = tsg.layer_norm_grad_workspace(rows, width)
        assert n > 0 and n % (2 * 4 * ((width + 7) // 8 * 8)) == 0
        assert n <= 2048 * 2 * 4 * ((width + 7) // 8 * 8)
    with pytest.raises(tsg.TsgemmError):
        tsg.layer_norm_grad_workspace(4, 0)


@pytest.mark.parametrize("call", ["quantize", "dequantize"])
@pytest.mark.parametrize("kw,needle", [
    (dict(rows=-1), ">= 0"),
    (dict(width=48), "divisible by 32"),
    (dict(dt=3), "dtype"),
    (dict(x=None), "NULL"),
    (dict(x=P + 1), "aligned"),
    (dict(ld=63), "row stride"),
    (dict(codes=None), "codes or scales"),
    (dict(codes=P + 4), "16-byte"),
    (dict(scales=P + 1), "4-byte"),
])
def test_mx_conversions_refuse(call, kw, needle):
    a = dict(rows=4, width=64, dt=B16, x=P, ld=64, codes=P, scales=P)
    a.update(kw)
    lib = tsg.load()
    if call == "quantize":
        rc = lib.tsgemm_mx_quantize(a["rows"], a["width"], a["dt"], a["x"], a["ld"], a["codes"], a["scales"], None)
    else:
        rc = lib.tsgemm_mx_dequantize(a["rows"], a["width"], a["dt"], a["codes"], a["scales"], a["x"], a["ld"], None)
    assert rc == tsg.EINVAL
    assert needle in tsg.last_error()


def _wgrad(rows=64, out=64, width=64, dt=B16, gdt=F32, dy=P, lddy=64, codes=P, scales=P, dw=P, ws=P, size=1 << 40):
    return tsg.load().tsgemm_mx_weight_grad(rows, out, width, dt, gdt, dy, lddy, codes, scales, dw, ws, size, None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(rows=-1), tsg.EINVAL, ">= 0"),
    (dict(out=-8), tsg.EINVAL, "out"),
    (dict(out=60), tsg.EINVAL, "divisible by 8"),
    (dict(width=40), tsg.EINVAL, "divisible by 32"),
    (dict(dt=F32), tsg.EINVAL, "dtype"),
    (dict(gdt=F16), tsg.EINVAL, "dw must be of"),
    (dict(dy=None), tsg.EINVAL, "dy is NULL"),
    (dict(dy=P + 8), tsg.EINVAL, "16-byte"),
    (dict(lddy=68), tsg.EINVAL, "16-byte"),
    (dict(lddy=56), tsg.EINVAL, "row stride"),
    (dict(lddy=1 << 24), tsg.EUNSUPPORTED, "2^24"),
    (dict(width=1 << 24), tsg.EUNSUPPORTED, "2^24"),
    (dict(codes=P + 8), tsg.EINVAL, "16-byte"),
    (dict(scales=None), tsg.EINVAL, "codes or scales"),
    (dict(dw=None), tsg.EINVAL, "dw"),
    (dict(dw=P + 4), tsg.EINVAL, "16-byte"),
    (dict(rows=65536, ws=None), tsg.EINVAL, "workspace"),
    (dict(rows=65536, ws=P + 8), tsg.EINVAL, "workspace"),
    (dict(rows=65536, size=16), tsg.EINVAL, "workspace"),
])
def test_weight_grad_refuses(kw, code, needle):
    assert _wgrad(**kw) == code
    assert needle in tsg.last_error()


def test_weight_grad_workspace():
    assert tsg.mx_weight_grad_workspace(8192, 0, 64) == 0
    assert tsg.mx_weight_grad_workspace(0, 64, 64) == 0
    assert tsg.mx_weight_grad_workspace(8192, 8192, 8192) == 0      # tiles enough: no split
    n = tsg.mx_weight_grad_workspace(65536, 64, 64)
    assert n > 0 and n % (4 * 64 * 64) == 0


def test_empty_calls_launch_nothing():
    assert _norm(rows=0, x=None, y=None) == tsg.OK
    assert _grad(rows=0, dy=None, x=None, dx=None, mean=None, rstd=None, dg=None, db=None, ws=None, size=0) == tsg.OK
    lib = tsg.load()
    for rows, width in ((0, 64), (4, 0)):
        assert lib.tsgemm_mx_quantize(rows, width, B16, None, 0, None, None, None) == tsg.OK
        assert lib.tsgemm_mx_dequantize(rows, width, B16, None, None, None, 0, None) == tsg.OK
    assert _wgrad(out=0, dy=None, dw=None) == tsg.OK
    assert _wgrad(width=0, codes=None, dw=None) == tsg.OK


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros((4, 64))
    v = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        tsg.layer_norm(x, v, v, 1e-5, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="two dimensions"):
        tsg.layer_norm(v, v, v, 1e-5, y=v)
    with pytest.raises(ValueError, match="CUDA"):
        tsg.layer_norm_grad(x, x, v, v, v, x)
    with pytest.raises(ValueError, match="CUDA"):
        tsg.mx_quantize(x, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        tsg.mx_dequantize(None, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        tsg.mx_weight_grad(x, None, None, torch.zeros((64, 64)))
    with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
        tsg.layer_norm(x.double(), v, v, 1e-5, y=x)


def test_extension_module_turns_down_what_the_binding_explains():
    """What the module does not take it leaves to the Python checks: None, no
    exception and no call."""
    with pytest.raises(ValueError):
        tsg.mx_quantize(torch.zeros((4, 64)), None, None)     # loads the module
    short = tsg._short
    x, v, b = torch.zeros((4, 64)), torch.zeros(64), torch.zeros((4, 64), dtype=torch.uint8)
    assert short.layer_norm(x, v, v, 1e-5, x, None, None, None, None) is None
    assert short.layer_norm(x, v, v) is None
    assert short.layer_norm(3, v, v, 1e-5, x, None, None, None, None) is None
    assert short.layer_norm_grad(x, x, v, v, v, x, None, None) is None
    assert short.mx_quantize(x, b, b) is None
    assert short.mx_quantize(None, None, None) is None
    assert short.mx_dequantize(x, b, b) is None
    assert short.mx_weight_grad(x, b, b, x) is None
    with pytest.raises(TypeError):
        short.setup(1, 2)
