"""What the tests of the gated projection and of the linear head's cross entropy
share: inputs, fp64 formulas and the bounds of their errors.

Bounds (derived, per element).  u = 2^-24 is the fp32 rounding, e the output
type's half step (bf16 2^-8, fp16 2^-11 relative; fp16 also 2^-25 absolute, its
subnormals' half step).
  * A product's fp32 sum of K terms: delta = 2 K u sum|terms| (every addition at
    most one unit in the last place off).
  * act is computed in fp32 from a g that is off by delta; |act'| <= 1.13, and the
    functions' own errors (exponentials of an argument that is itself rounded:
    |g| <= 64 times u log2 e, a division, a few products) stay below 2^-17 |act(g)| + 2^-22.
    y = act(g) u is off by e |y| + 1.13 delta_g |u| + (|act| + 1.13 delta_g) delta_u
    + 2^-17 |y| + 2^-22 |u|.
  * dg and du are rounded to the type and come from functions as above:
    (e + 2^-16) |dg| + 2^-20 |dy up| each, the last term for slopes near their zero;
    fp16 adds 2^-25.  The products add these up: dx is off by
    e |dx| + sum of those |weight| + delta of the product.
  * lse: the largest delta of the row's logits, 2^-17 for the sum of exponentials
    (at most 128 additions on any way, u each, and exponents off by 2 u |l| log2 e),
    2^-21 max|l|, and u |lse|; loss adds the target's delta and u |loss|.
  * dl: |dloss| (p (delta + 2^-18 + 2^-21 max|l|) + (e + 2^-20) |p - onehot|); in fp16 the
    scaled subnormals add 2^-25 2^-13 2 max|dloss|.  dx and dweight as above.
"""

import math

import torch

DEV = torch.device("cuda:0")
U = 2.0 ** -24
FP16, BF16 = torch.float16, torch.bfloat16
ACTS = ("silu", "gelu", "gelu_tanh")


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return 2.0 ** -25 if t == FP16 else 0.0


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(DEV)


def act64(name, g):
    """act(g) and its derivative in fp64."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    if name == "gelu":
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def product(a, b):
    """a b^T in fp64 and the bound of its fp32 sum."""
    a, b = a.double(), b.double()
    return a @ b.t(), 2 * a.shape[1] * U * (a.abs() @ b.abs().t())


def check(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got - want).abs()
    bad = (err > bound).sum().item()
    assert bad == 0, f"{what}: {bad} of {got.numel()} outside, worst {(err / bound.clamp_min(1e-300)).max().item():.3g} of the bound"


def gated_inputs(rows, width, hidden, dtype, seed):
    x = randn(seed, rows, width).to(dtype)
    return x, randn(seed + 1, hidden, width, scale=1.2 * width ** -0.5).to(dtype), randn(seed + 2, hidden, width, scale=width ** -0.5).to(dtype)


def check_gated(x, wg, wu, act, y, gate, up, what):
    e, t = half(x.dtype), tiny(x.dtype)
    g, dg = product(x, wg)
    u, du = product(x, wu)
    a, _ = act64(act, g)
    check(y, a * u, e * (a * u).abs() + 1.13 * dg * u.abs() + (a.abs() + 1.13 * dg) * du + 2.0 ** -17 * (a * u).abs() + 2.0 ** -22 * u.abs() + t, what + " y")
    if gate is not None:
        check(gate, g, (e + U) * g.abs() + dg + t, what + " gate")
    if up is not None:
        check(up, u, (e + U) * u.abs() + du + t, what + " up")


def check_gated_grad(dy, x, wg, wu, gate, up, act, dx, dwg, dwu, what):
    e, t = half(x.dtype), tiny(x.dtype)
    a, slope = act64(act, gate.double())
    dy, u = dy.double(), up.double()
    dg, du = dy * u * slope, dy * a
    off_g = (e + 2.0 ** -16) * dg.abs() + 2.0 ** -20 * (dy * u).abs() + t
    off_u = (e + 2.0 ** -16) * du.abs() + 2.0 ** -20 * dy.abs() + t
    if dx is not None:
        want = dg @ wg.double() + du @ wu.double()
        bound = (off_g + 4 * dg.shape[1] * U * dg.abs()) @ wg.double().abs() + (off_u + 4 * dg.shape[1] * U * du.abs()) @ wu.double().abs()
        check(dx, want, e * want.abs() + bound + t, what + " dx")
    if dwg is not None:
        n = 2 * x.shape[0] * U
        for got, d, off, name in ((dwg, dg, off_g, "dgate_weight"), (dwu, du, off_u, "dup_weight")):
            want = d.t() @ x.double()
            check(got, want, e * want.abs() + (off + n * d.abs()).t() @ x.double().abs() + t, f"{what} {name}")


def loss_inputs(rows, width, vocab, dtype, seed, ignored=0.2, ignore=-100):
    w = randn(seed, vocab, width, scale=2 * width ** -0.5).to(dtype)
    g = torch.Generator().manual_seed(seed + 1)
    target = torch.randint(0, vocab, (rows,), generator=g).to(DEV)
    x = (randn(seed + 2, rows, width) + 2 * (torch.rand((rows, 1), generator=g) < 0.5).to(DEV).float() * w[target].float()).to(dtype)
    target[(torch.rand(rows, generator=g) < ignored).to(DEV)] = ignore
    return x, w, target


def loss64(x, w, target, ignore=-100):
    l, delta = product(x, w)
    lse = torch.logsumexp(l, dim=1)
    hit = l.gather(1, target.clamp(0, w.shape[0] - 1)[:, None])[:, 0]
    return torch.where(target == ignore, 0.0, lse - hit), lse, l, delta


def check_loss(x, w, target, loss, lse, what, ignore=-100):
    want, want_lse, l, delta = loss64(x, w, target, ignore)
    off = delta.amax(dim=1)
    b = off + 2.0 ** -17 + 2.0 ** -21 * l.abs().amax(dim=1) + U * want_lse.abs()
    check(lse, want_lse, b, what + " lse")
    check(loss, want, torch.where(target == ignore, 0.0, b + off + U * want.abs()), what + " loss")


def check_loss_grad(dloss, x, w, target, lse, dx, dw, what, ignore=-100):
    e, t = half(x.dtype), tiny(x.dtype)
    l, delta = product(x, w)
    counted = target != ignore
    p = torch.exp(l - lse.double()[:, None])
    d = torch.where(counted, dloss.double(), 0.0)[:, None]
    dl = p.clone()
    at = torch.nonzero(counted)[:, 0]
    dl[at, target[at]] -= 1.0
    off = d.abs() * (p * (delta + 2.0 ** -18 + 2.0 ** -21 * l.abs().amax(dim=1, keepdim=True)) + (e + 2.0 ** -20) * dl.abs())
    if x.dtype == FP16:
        off = off + 2.0 ** -37 * d.abs().max()
    dl = dl * d
    if dx is not None:
        want = dl @ w.double()
        check(dx, want, e * want.abs() + (off + 2 * (w.shape[0] + 64) * U * dl.abs()) @ w.double().abs() + t, what + " dx")
    if dw is not None:
        xc = torch.where(counted[:, None], x.double(), 0.0)
        want = dl.t() @ xc
        check(dw, want, e * want.abs() + (off + 2 * (x.shape[0] + 64) * U * dl.abs()).t() @ xc.abs() + t, what + " dweight")
