"""The gated projection, the cross entropy of a linear head and their gradients where
they can go wrong: views and odd addresses, rows that do not count, targets outside
the vocabulary, empty calls, streams, captured graphs, offsets past 32 bits,
differences, and all of them together in one training step.  Bounds: linear_cases.py."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg
from tests.linear_cases import (ACTS, BF16, DEV, FP16, U, act64, check, check_gated, check_gated_grad, check_loss, check_loss_grad, gated_inputs,
                                half, loss64, loss_inputs, randn)

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)


def nan(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def view(rows, width, ld, offset, dtype):
    """A view with its buffer, all NaN."""
    buf = nan(offset + rows * ld + 16, dtype=dtype)
    return buf[offset: offset + rows * ld].view(rows, ld)[:, :width], buf


def holds_only(v, buf, offset, rows, width, ld):
    """Nothing but the view was written."""
    rest = buf.clone()
    rest[offset: offset + rows * ld].view(rows, ld)[:, :width] = float("nan")
    assert torch.isnan(rest.float()).all()


@DTYPES
@pytest.mark.parametrize("rows,width,hidden", [(5, 72, 37), (70, 136, 131), (300, 72, 515), (2049, 72, 4099)])
def test_views_and_odd_addresses(dtype, rows, width, hidden):
    x, wg, wu = gated_inputs(rows, width, hidden, dtype, 3)
    dy = randn(4, rows, hidden, scale=0.1).to(dtype)
    packed = [nan(rows, hidden, dtype=dtype) for _ in range(3)]
    tsg.gated_linear(x, wg, wu, packed[0], "gelu", gate=packed[1], up=packed[2])
    xs, ws, us = (view(*t.shape, width + pad, 8 * k, dtype)[0].copy_(t) for k, (t, pad) in enumerate(((x, 8), (wg, 24), (wu, 16))))
    for ld, offset in ((hidden, 0), (hidden + 1, 1), (hidden + 8, 8), (hidden + 5, 3)):
        outs = [view(rows, hidden, ld + k, offset, dtype) for k in range(3)]
        tsg.gated_linear(xs, ws, us, outs[0][0], "gelu", gate=outs[1][0], up=outs[2][0])
        for k, (o, buf) in enumerate(outs):
            assert torch.equal(o, packed[k]), (ld, offset, k)
            holds_only(o, buf, offset, rows, hidden, ld + k)
        dys = view(rows, hidden, ld + 2, offset, dtype)[0].copy_(dy)
        want = nan(rows, width, dtype=dtype), nan(hidden, width, dtype=dtype), nan(hidden, width, dtype=dtype)
        tsg.gated_linear_grad(dy, x, wg, wu, packed[1], packed[2], *want, "gelu")
        got = view(rows, width, width + 8, 8, dtype), view(hidden, width, width + 16, 0, dtype), view(hidden, width, width + 8, 16, dtype)
        tsg.gated_linear_grad(dys, xs, ws, us, outs[1][0], outs[2][0], *(g[0] for g in got), "gelu")
        for w, (g, buf), at, d in zip(want, got, (8, 0, 16), (8, 16, 8)):
            assert torch.equal(w, g)
            holds_only(g, buf, at, g.shape[0], width, width + d)


@DTYPES
def test_loss_views(dtype):
    rows, width, vocab = 130, 136, 1003
    x, w, target = loss_inputs(rows, width, vocab, dtype, 5)
    xs, ws = view(rows, width, width + 16, 8, dtype)[0].copy_(x), view(vocab, width, width + 8, 0, dtype)[0].copy_(w)
    a, b = [nan(rows) for _ in range(2)], [nan(rows) for _ in range(2)]
    tsg.linear_cross_entropy(x, w, target, *a)
    tsg.linear_cross_entropy(xs, ws, target, *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dloss = randn(6, rows)
    dx, dw = nan(rows, width, dtype=dtype), nan(vocab, width, dtype=dtype)
    tsg.linear_cross_entropy_grad(dloss, x, w, target, a[1], dx, dw)
    (ex, bx), (ew, bw) = view(rows, width, width + 24, 16, dtype), view(vocab, width, width + 8, 8, dtype)
    tsg.linear_cross_entropy_grad(dloss, xs, ws, target, a[1], ex, ew)
    assert torch.equal(dx, ex) and torch.equal(dw, ew)
    holds_only(ex, bx, 16, rows, width, width + 24)
    holds_only(ew, bw, 8, vocab, width, width + 8)


@DTYPES
@pytest.mark.parametrize("rows,width,vocab", [(20, 72, 300), (140, 136, 1003), (2049, 72, 8200)])
def test_rows_that_do_not_count(dtype, rows, width, vocab):
    """NaN and infinities in ignored rows reach nothing; a vocabulary index may be the ignored one."""
    x, w, target = loss_inputs(rows, width, vocab, dtype, 7, ignored=0.4, ignore=3)
    out = target == 3
    assert out.any() and not out.all()
    loss, lse = nan(rows), nan(rows)
    tsg.linear_cross_entropy(x, w, target, loss, lse, ignore_index=3)
    check_loss(x, w, target, loss, lse, "ignored 3", ignore=3)
    dloss = randn(8, rows)
    want = nan(rows, width, dtype=dtype), nan(vocab, width, dtype=dtype)
    tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, *want, ignore_index=3)
    check_loss_grad(dloss, x, w, target, lse, *want, "ignored 3", ignore=3)
    bad = x.clone()
    bad[out] = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min], dtype=dtype, device=DEV).repeat(width // 4)
    l2, s2 = nan(rows), nan(rows)
    tsg.linear_cross_entropy(bad, w, target, l2, s2, ignore_index=3)
    assert torch.equal(l2, loss) and torch.equal(s2[~out], lse[~out])
    got = nan(rows, width, dtype=dtype), nan(vocab, width, dtype=dtype)
    tsg.linear_cross_entropy_grad(torch.where(out, float("nan"), dloss), bad, w, target, torch.where(out, float("inf"), lse), *got, ignore_index=3)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not got[0][out].any()


@DTYPES
def test_targets_outside_the_vocabulary(dtype):
    rows, width, vocab = 40, 72, 300
    for n in (rows, 20):
        x, w, target = loss_inputs(n, width, vocab, dtype, 9, ignored=0.0)
        for i, t in enumerate((-1, vocab, vocab + 1, 1 << 40, -(1 << 40), (1 << 32) + 5, -99)):
            target[2 * i] = t
        bad = (target < 0) | (target >= vocab)
        loss, lse = nan(n), nan(n)
        tsg.linear_cross_entropy(x, w, target, loss, lse)
        assert torch.equal(torch.isnan(loss), bad) and torch.isfinite(lse).all()
        masked = torch.where(bad, -100, target)
        dloss = randn(1, n)
        a, b = ((nan(n, width, dtype=dtype), nan(vocab, width, dtype=dtype)) for _ in range(2))
        tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, *a)
        tsg.linear_cross_entropy_grad(dloss, x, w, masked, lse, *b)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and not a[0][bad].any()


@DTYPES
def test_nothing_counts(dtype):
    rows, width, vocab = 70, 72, 300
    x, w, target = loss_inputs(rows, width, vocab, dtype, 9)
    lse = loss64(x, w, target)[1].float()
    for t, d in ((torch.full_like(target, -100), randn(1, rows)), (target, torch.zeros(rows, device=DEV))):
        loss, s = nan(rows), nan(rows)
        tsg.linear_cross_entropy(x, w, t, loss, s)
        check_loss(x, w, t, loss, s, "nothing counts")
        dx, dw = nan(rows, width, dtype=dtype), nan(vocab, width, dtype=dtype)
        tsg.linear_cross_entropy_grad(d, x, w, t, lse, dx, dw)
        assert not dx.any() and not dw.any()


@DTYPES
@pytest.mark.parametrize("rows", [7, 100])
def test_far_logits_and_no_numbers(dtype, rows):
    """Logits of thousands, rows of equal ones, rows with a NaN or an infinity."""
    width, vocab = 64, 515
    x, w, target = loss_inputs(rows, width, vocab, dtype, 11, ignored=0.0)
    x *= 200
    x[1] = 0
    loss, lse = nan(rows), nan(rows)
    tsg.linear_cross_entropy(x, w, target, loss, lse)
    check_loss(x, w, target, loss, lse, "far")
    x[2, 5], x[4, 7] = float("nan"), float("inf")
    l2, s2 = nan(rows), nan(rows)
    tsg.linear_cross_entropy(x, w, target, l2, s2)
    rest = torch.ones(rows, dtype=torch.bool, device=DEV)
    rest[2] = rest[4] = False
    assert torch.isnan(l2[~rest]).all() and torch.isnan(s2[~rest]).all()
    assert torch.equal(l2[rest], loss[rest]) and torch.equal(s2[rest], lse[rest])


@DTYPES
def test_uneven_dloss(dtype):
    """Rows whose dloss differ by many orders of magnitude, negative ones too."""
    rows, width, vocab = 150, 136, 700
    x, w, target = loss_inputs(rows, width, vocab, dtype, 12)
    lse = loss64(x, w, target)[1].float()
    dloss = randn(2, rows) * torch.exp2(torch.arange(rows, device=DEV) % 24 - 16.0)
    dx, dw = nan(rows, width, dtype=dtype), nan(vocab, width, dtype=dtype)
    tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, dx, dw)
    check_loss_grad(dloss, x, w, target, lse, dx, dw, "uneven")


@pytest.mark.parametrize("act", ACTS)
def test_far_activations(act):
    """Projections far out on either side: the activations end in 0 and in g, their slopes in 0 and 1."""
    rows, width, hidden = 40, 64, 128
    x, wg, wu = gated_inputs(rows, width, hidden, BF16, 13)
    x *= 30
    for n in (rows, 9):
        y, gate, up = (nan(n, hidden, dtype=BF16) for _ in range(3))
        tsg.gated_linear(x[:n], wg, wu, y, act, gate=gate, up=up)
        check_gated(x[:n], wg, wu, act, y, gate, up, "far")
    gate = torch.linspace(-60, 60, rows * hidden, device=DEV).view(rows, hidden).to(BF16)
    dy, dx, dwg, dwu = randn(1, rows, hidden).to(BF16), nan(rows, width, dtype=BF16), nan(hidden, width, dtype=BF16), nan(hidden, width, dtype=BF16)
    up = randn(2, rows, hidden).to(BF16)
    tsg.gated_linear_grad(dy, x, wg, wu, gate, up, dx, dwg, dwu, act)
    check_gated_grad(dy, x, wg, wu, gate, up, act, dx, dwg, dwu, "far")


@DTYPES
def test_empty_calls(dtype):
    e = lambda *s: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    i64, f32 = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    tsg.gated_linear(e(0, 64), e(8, 64), e(8, 64), e(0, 8))
    tsg.gated_linear(e(8, 64), e(0, 64), e(0, 64), e(8, 0))
    dx, dg, du = nan(0, 64, dtype=dtype), nan(8, 64, dtype=dtype), nan(8, 64, dtype=dtype)
    tsg.gated_linear_grad(e(0, 8), e(0, 64), e(8, 64), e(8, 64), e(0, 8), e(0, 8), dx, dg, du)
    assert not dg.any() and not du.any()
    dx = nan(8, 64, dtype=dtype)
    tsg.gated_linear_grad(e(8, 0), e(8, 64), e(0, 64), e(0, 64), e(8, 0), e(8, 0), dx, e(0, 64), e(0, 64))
    assert not dx.any()
    tsg.linear_cross_entropy(e(0, 64), e(9, 64), i64, f32, f32.clone())
    dw = nan(9, 64, dtype=dtype)
    tsg.linear_cross_entropy_grad(f32, e(0, 64), e(9, 64), i64, f32.clone(), e(0, 64), dw)
    assert not dw.any()


def test_in_place_is_refused():
    x, wg, wu = gated_inputs(64, 64, 64, BF16, 1)
    y = nan(64, 64, dtype=BF16)
    with pytest.raises(tsg.TsgemmError, match="overlaps"):
        tsg.gated_linear(x, wg, wu, x)
    with pytest.raises(tsg.TsgemmError, match="overlaps"):
        tsg.gated_linear_grad(y, x, wg, wu, y, y, dx=y)
    with pytest.raises(tsg.TsgemmError, match="workspace"):
        tsg.gated_linear_grad(y, x, wg, wu, y, y, dx=y.clone(), workspace=torch.empty(16, device=DEV))


def everything(t, o, stream=None, ws=None):
    ws = ws or {}
    tsg.gated_linear(t["x"], t["wg"], t["wu"], o["y"], gate=o["gate"], up=o["up"], stream=stream)
    tsg.gated_linear_grad(t["dy"], t["x"], t["wg"], t["wu"], o["gate"], o["up"], o["dx"], o["dwg"], o["dwu"], stream=stream, workspace=ws.get("gg"))
    tsg.linear_cross_entropy(t["x"], t["w"], t["target"], o["loss"], o["lse"], stream=stream, workspace=ws.get("l"))
    tsg.linear_cross_entropy_grad(t["dloss"], t["x"], t["w"], t["target"], o["lse"], o["ex"], o["dw"], stream=stream, workspace=ws.get("lg"))


def tensors(rows, width, hidden, vocab, dtype, seed):
    x, wg, wu = gated_inputs(rows, width, hidden, dtype, seed)
    _, w, target = loss_inputs(rows, width, vocab, dtype, seed + 5)
    return {"x": x, "wg": wg, "wu": wu, "w": w, "target": target, "dy": randn(seed + 9, rows, hidden, scale=0.1).to(dtype), "dloss": randn(seed + 10, rows)}


def outputs(rows, width, hidden, vocab, dtype):
    n = lambda *s: nan(*s, dtype=dtype)  # noqa: E731
    return {"y": n(rows, hidden), "gate": n(rows, hidden), "up": n(rows, hidden), "dx": n(rows, width), "dwg": n(hidden, width), "dwu": n(hidden, width),
            "loss": nan(rows), "lse": nan(rows), "ex": n(rows, width), "dw": n(vocab, width)}


SIZES = [(1, 264, 300, 1003), (30, 264, 300, 1003), (700, 264, 1300, 5003)]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_streams(sizes):
    """Two streams at once, each with the work of the other's; workspaces of torch's allocator."""
    sets = [tensors(*sizes, BF16, s) for s in (20, 40)]
    want = [outputs(*sizes, BF16) for _ in sets]
    for t, o in zip(sets, want):
        everything(t, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [outputs(*sizes, BF16) for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        for t, o, s in zip(sets, got, streams):
            everything(t, o, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for name in a:
            assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_two_captured_graphs(sizes):
    """Two graphs with workspaces of their own, replayed in turn with changed inputs and eager work between."""
    rows, width, hidden, vocab = sizes
    need = {"gg": tsg.gated_linear_grad_workspace(rows, hidden, width), "l": tsg.linear_cross_entropy_workspace(rows, vocab, width),
            "lg": tsg.linear_cross_entropy_grad_workspace(rows, vocab, width)}
    graphs = []
    for k in range(2):
        t, o = tensors(*sizes, FP16, 60 + k), outputs(*sizes, FP16)
        ws = {name: torch.empty(n, dtype=torch.uint8, device=DEV) for name, n in need.items()} if k else None
        everything(t, o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            everything(t, o, ws=ws)
        graphs.append((g, t, o, ws))
    for i in range(4):
        for k, (g, t, o, _) in enumerate(graphs):
            for name, v in tensors(*sizes, FP16, 100 + 10 * i + k).items():
                t[name].copy_(v)
            for v in o.values():
                v.fill_(float("nan"))
        for g, _, _, _ in graphs:
            g.replay()
        eager = [outputs(*sizes, FP16) for _ in graphs]
        for (_, t, _, _), e in zip(graphs, eager):
            everything(t, e)
        torch.cuda.synchronize()
        for (_, _, o, _), e in zip(graphs, eager):
            for name in e:
                assert torch.equal(o[name], e[name]), (i, name)


def test_same_bits_every_time():
    t, first = tensors(1500, 520, 2000, 9000, BF16, 3), outputs(1500, 520, 2000, 9000, BF16)
    everything(t, first)
    for _ in range(5):
        o = outputs(1500, 520, 2000, 9000, BF16)
        everything(t, o)
        for name in o:
            assert torch.equal(o[name], first[name]), name


def test_offsets_past_32_bits():
    """A weight and its gradient of 4.6 GB, and y with rows 3 MB apart over 6.3 GB."""
    rows, width, vocab = 40, 4096, 560001
    w = torch.empty((vocab, width), dtype=BF16, device=DEV)
    for i in range(0, vocab, 1 << 16):
        w[i: i + (1 << 16)] = torch.randn(w[i: i + (1 << 16)].shape, device=DEV) * (2 * width ** -0.5)
    x, target = randn(1, rows, width).to(BF16), torch.randint(0, vocab, (rows,), device=DEV)
    target[:4] = torch.tensor([vocab - 1, vocab - 2, 0, vocab - 300], device=DEV)
    for n in (rows, 20):
        loss, lse = nan(n), nan(n)
        tsg.linear_cross_entropy(x[:n], w, target[:n], loss, lse)
        l = torch.cat([x[:n].double() @ w[i: i + (1 << 16)].double().t() for i in range(0, vocab, 1 << 16)], dim=1)
        want = torch.logsumexp(l, dim=1)
        # 2 K u sum|terms| of the logits, below 2^-8 here; the rest as in linear_cases.py
        assert ((lse - want).abs() < 2.0 ** -8).all()
        assert ((loss - (want - l.gather(1, target[:n, None])[:, 0])).abs() < 2.0 ** -7).all()
    dx, dw = nan(rows, width, dtype=BF16), nan(vocab, width, dtype=BF16)
    dloss = torch.full((rows,), 1.0 / rows, device=DEV)
    l = torch.cat([x.double() @ w[i: i + (1 << 16)].double().t() for i in range(0, vocab, 1 << 16)], dim=1)
    lse = torch.logsumexp(l, dim=1).float()
    tsg.linear_cross_entropy_grad(dloss, x, w, target, lse, dx, dw)
    d = torch.exp(l - lse[:, None].double()) / rows
    d[torch.arange(rows, device=DEV), target] -= 1.0 / rows
    for at in (slice(0, 300), slice(524200, 524600), slice(vocab - 600, vocab)):
        part = d[:, at].t()
        bound = (half(BF16) + 2.0 ** -6) * (part.abs() @ x.double().abs())
        check(dw[at], part @ x.double(), bound + half(BF16) * (part @ x.double()).abs(), "dweight")
    want = sum(d[:, i: i + (1 << 16)] @ w[i: i + (1 << 16)].double() for i in range(0, vocab, 1 << 16))
    assert (dx.double() - want).norm() <= 2.0 ** -7 * want.norm()
    del w, dw, l, d
    torch.cuda.empty_cache()
    rows, width, hidden, ld = 2100, 64, 300, 1500001
    a, wg, wu = gated_inputs(rows, width, hidden, BF16, 2)
    buf = torch.zeros(rows * ld, dtype=BF16, device=DEV)
    y = buf.view(rows, ld)[:, :hidden]
    tsg.gated_linear(a, wg, wu, y)
    check_gated(a, wg, wu, "silu", y.contiguous(), None, None, "far rows")
    y.fill_(0)
    assert not buf.any()


def test_gradients_against_differences():
    """Central differences of the fp64 formulas along random directions: their own error is
    h^2 / 6 times the third derivative, below 1e-6 of the sums here; the kernel's gradients are
    off by e and a half step of dl, dg and du, each relative to the magnitudes summed."""
    rows, width, hidden, vocab = 50, 72, 90, 200
    x, w, target = loss_inputs(rows, width, vocab, BF16, 21)
    dloss, h = randn(3, rows), 1e-4
    dx, dw = nan(rows, width, dtype=BF16), nan(vocab, width, dtype=BF16)
    tsg.linear_cross_entropy_grad(dloss, x, w, target, loss64(x, w, target)[1].float(), dx, dw)
    f = lambda a, b: (dloss.double() * loss64(a, b, target)[0]).sum()  # noqa: E731
    dirx, dirw = randn(4, rows, width).double(), randn(5, vocab, width).double()
    for got, d, diff in ((dx, dirx, (f(x.double() + h * dirx, w) - f(x.double() - h * dirx, w)) / (2 * h)),
                         (dw, dirw, (f(x, w.double() + h * dirw) - f(x, w.double() - h * dirw)) / (2 * h))):
        assert (got.double() * d).sum().sub(diff).abs() <= 3 * half(BF16) * (got.double() * d).abs().sum() + 1e-6 * (got.double() * d).abs().sum()
    for act in ACTS:
        x, wg, wu = gated_inputs(rows, width, hidden, BF16, 22)
        dy = randn(6, rows, hidden).to(BF16)
        gate, up = (nan(rows, hidden, dtype=BF16) for _ in range(2))
        tsg.gated_linear(x, wg, wu, torch.empty_like(gate), act, gate=gate, up=up)
        dx, dg, du = nan(rows, width, dtype=BF16), nan(hidden, width, dtype=BF16), nan(hidden, width, dtype=BF16)
        tsg.gated_linear_grad(dy, x, wg, wu, gate, up, dx, dg, du, act)
        f = lambda a, b, c: (dy.double() * act64(act, a.double() @ b.double().t())[0] * (a.double() @ c.double().t())).sum()  # noqa: E731
        args = [x.double(), wg.double(), wu.double()]
        for i, got in enumerate((dx, dg, du)):
            d = randn(7 + i, *got.shape).double()
            up_, down = list(args), list(args)
            up_[i], down[i] = args[i] + h * d, args[i] - h * d
            diff = (f(*up_) - f(*down)) / (2 * h)
            # gate and up are rounded too: their half steps times |g act''| and |act'| <= 1.2 enter the same sums
            assert (got.double() * d).sum().sub(diff).abs() <= 6 * half(BF16) * (got.double() * d).abs().sum() + 1e-6, (act, i)


def test_one_training_step_together():
    """Layer norm, the gated projection, the product that leads back, the linear head's cross
    entropy, and all of their gradients: every call against its formula on the tensors that the
    step gave it, and the loss against fp64 throughout."""
    rows, width, hidden, vocab, dt = 384, 256, 640, 3001, BF16
    e = half(dt)
    x = randn(1, rows, width).to(dt)
    gamma, beta = (1 + 0.1 * randn(2, width)), 0.1 * randn(3, width)
    wg, wu = randn(4, hidden, width, scale=1.2 * width ** -0.5).to(dt), randn(5, hidden, width, scale=width ** -0.5).to(dt)
    down, head = randn(6, hidden, width, scale=hidden ** -0.5).to(dt), randn(7, vocab, width, scale=2 * width ** -0.5).to(dt)
    target = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(8)).to(DEV)
    target[::9] = -100
    n, mean, rstd = nan(rows, width, dtype=dt), nan(rows), nan(rows)
    tsg.layer_norm(x, gamma, beta, 1e-5, y=n, mean=mean, rstd=rstd)
    y, gate, up, z = nan(rows, hidden, dtype=dt), nan(rows, hidden, dtype=dt), nan(rows, hidden, dtype=dt), nan(rows, width, dtype=dt)
    tsg.gated_linear(n, wg, wu, y, gate=gate, up=up)
    check_gated(n, wg, wu, "silu", y, gate, up, "step")
    tsg.Plan(rows, width, hidden, "bf16", 128, 128, 64, 8, 2).run(y, down, z)
    loss, lse = nan(rows), nan(rows)
    tsg.linear_cross_entropy(z, head, target, loss, lse)
    check_loss(z, head, target, loss, lse, "step")
    counted = (target != -100).float()
    dloss = counted / counted.sum()
    dz, dhead = nan(rows, width, dtype=dt), nan(vocab, width, dtype=dt)
    tsg.linear_cross_entropy_grad(dloss, z, head, target, lse, dz, dhead)
    check_loss_grad(dloss, z, head, target, lse, dz, dhead, "step")
    dy = nan(rows, hidden, dtype=dt)
    tsg.Plan(rows, hidden, width, "bf16", 128, 128, 64, 8, 2).run(dz, down.t().contiguous(), dy)
    dn, dwg, dwu = nan(rows, width, dtype=dt), nan(hidden, width, dtype=dt), nan(hidden, width, dtype=dt)
    tsg.gated_linear_grad(dy, n, wg, wu, gate, up, dn, dwg, dwu)
    check_gated_grad(dy, n, wg, wu, gate, up, "silu", dn, dwg, dwu, "step")
    dx, dgamma, dbeta = nan(rows, width, dtype=dt), nan(width), nan(width)
    tsg.layer_norm_grad(dn, x, gamma, mean, rstd, dx, dgamma, dbeta)
    leaves = [t.double().requires_grad_() for t in (x, gamma, beta, wg, wu, down, head)]
    a, ga, be, g64, u64, d64, h64 = leaves
    m = (a - a.mean(dim=1, keepdim=True)) * (a.var(dim=1, unbiased=False, keepdim=True) + 1e-5).rsqrt() * ga + be
    gt = m @ g64.t()
    logits = ((gt * torch.sigmoid(gt)) * (m @ u64.t())) @ d64 @ h64.t()
    total = torch.nn.functional.cross_entropy(logits, target, ignore_index=-100)
    total.backward()
    # four roundings on the way forward and six back, each at most e of its tensor, whose effects on
    # a sum of hundreds of terms of either sign add up like their squares: below 4 e of the norms
    assert abs((loss * dloss).sum().item() - total.item()) <= 4 * e * abs(total.item())
    for got, leaf in ((dx, a), (dgamma, ga), (dbeta, be), (dwg, g64), (dwu, u64), (dhead, h64)):
        assert (got.double() - leaf.grad).norm() <= 4 * e * leaf.grad.norm()
