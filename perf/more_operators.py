"""What is measured of the operators around a language model's linear layers: the
gated feed-forward projection y = act(x Wg^T) * (x Wu^T) with its gradient, and
the softmax cross entropy of a linear head over a large vocabulary, whose logits
are not kept, with its gradient.

A case is one call.  `run` makes it either through the library (`own`) or in
its plain form: elementary torch operations in fp32, rounded once at the end.
`exact` gives the same outputs from the definitions in fp64.
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100
MOST_GATED = 8192 * 4096 * 16384    # rows * width * hidden
MOST_LOSS = 8192 * 4096 * 131072    # rows * width * vocab


def listed():
    return [
        # one token's feed-forward layer while a model answers: the weights' way through the chip
        {"name": "gated one token bf16", "op": "gated", "rows": 1, "width": 4096, "hidden": 8192, "dtype": "bf16", "act": "silu", "keep": False},
        # a ragged batch of prompts (rows, width and hidden that no tile divides)
        {"name": "gated ragged fp16", "op": "gated", "rows": 1000, "width": 2504, "hidden": 6001, "dtype": "fp16", "act": "gelu", "keep": False},
        # a training batch, both projections kept for the backward pass
        {"name": "gated batch bf16", "op": "gated", "rows": 8192, "width": 4096, "hidden": 16384, "dtype": "bf16", "act": "silu", "keep": True},
        # a small model's backward pass: latency
        {"name": "gated grad small fp16", "op": "gated_grad", "rows": 512, "width": 512, "hidden": 1024, "dtype": "fp16", "act": "silu"},
        # a ragged backward pass
        {"name": "gated grad ragged bf16", "op": "gated_grad", "rows": 4000, "width": 2504, "hidden": 6001, "dtype": "bf16", "act": "gelu_tanh"},
        # a training batch's backward pass
        {"name": "gated grad batch bf16", "op": "gated_grad", "rows": 8192, "width": 4096, "hidden": 16384, "dtype": "bf16", "act": "silu"},
        # a few answers scored: the head's weight once through the chip
        {"name": "loss 16 rows bf16", "op": "loss", "rows": 16, "width": 4096, "vocab": 131072, "dtype": "bf16", "ignored": 0.0},
        # a fine-tuning batch: prompts masked out, an odd vocabulary
        {"name": "loss ragged fp16", "op": "loss", "rows": 1000, "width": 1000, "vocab": 50001, "dtype": "fp16", "ignored": 0.4},
        # a training batch over a large vocabulary
        {"name": "loss batch bf16", "op": "loss", "rows": 8192, "width": 4096, "vocab": 131072, "dtype": "bf16", "ignored": 0.05},
        # a small model's backward pass: latency
        {"name": "loss grad small fp16", "op": "loss_grad", "rows": 512, "width": 512, "vocab": 8192, "dtype": "fp16", "ignored": 0.05},
        # a fine-tuning batch's backward pass
        {"name": "loss grad ragged bf16", "op": "loss_grad", "rows": 2000, "width": 2504, "vocab": 50001, "dtype": "bf16", "ignored": 0.4},
        # a training batch's backward pass
        {"name": "loss grad batch bf16", "op": "loss_grad", "rows": 8192, "width": 4096, "vocab": 131072, "dtype": "bf16", "ignored": 0.05},
    ]


def draw(rng):
    def size(low, high, step=1):
        v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        return max(low, min(high, v // step * step))

    op = rng.choice(("gated", "gated_grad", "loss", "loss_grad"))
    case = {"op": op, "width": size(64, 8192, rng.choice((8, 8, 64))), "dtype": rng.choice(("fp16", "bf16"))}
    if op in ("gated", "gated_grad"):
        case["hidden"] = size(64, 16384, rng.choice((1, 8, 64)))
        case["rows"] = size(1, min(16384, MOST_GATED // (case["width"] * case["hidden"])))
        case["act"] = rng.choice(("silu", "gelu", "gelu_tanh"))
        if op == "gated":
            case["keep"] = rng.random() < 0.5
    else:
        case["vocab"] = size(512, 131072, rng.choice((1, 8, 64)))
        case["rows"] = size(1, min(16384, MOST_LOSS // (case["width"] * case["vocab"])))
        case["ignored"] = rng.choice((0.0, 0.05, 0.4))
    return case


def work(case):
    rows, width = case["rows"], case["width"]
    if case["op"] == "gated":
        hidden = case["hidden"]
        return {"bytes": 2 * (rows * width + 2 * hidden * width + rows * hidden * (3 if case["keep"] else 1)),
                "flops": 4 * rows * width * hidden}
    if case["op"] == "gated_grad":
        hidden = case["hidden"]
        return {"bytes": 2 * (3 * rows * hidden + 2 * rows * width + 4 * hidden * width), "flops": 8 * rows * width * hidden}
    vocab = case["vocab"]
    if case["op"] == "loss":
        return {"bytes": 2 * (rows * width + vocab * width) + 16 * rows, "flops": 2 * rows * width * vocab}
    return {"bytes": 4 * (rows * width + vocab * width) + 16 * rows, "flops": 6 * rows * width * vocab}


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows, width, dtype = case["rows"], case["width"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # normalised hidden states: channels of different size, a few of them larger
    spread = torch.exp(0.3 * normal(width))
    spread = torch.where(torch.rand(width, generator=g, device=dev) < 0.01, 4 * spread, spread)
    x = normal(rows, width) * spread
    s = {"case": dict(case)}
    if case["op"] in ("gated", "gated_grad"):
        hidden = case["hidden"]
        s["x"] = x.to(dtype)
        s["gate_weight"] = (1.2 * width ** -0.5 * normal(hidden, width)).to(dtype)
        s["up_weight"] = (width ** -0.5 * normal(hidden, width)).to(dtype)
        if case["op"] == "gated":
            for name in ("y", "gate", "up") if case["keep"] else ("y",):
                s[name] = torch.empty((rows, hidden), dtype=dtype, device=dev)
            return s
        s["gate"] = (s["x"].float() @ s["gate_weight"].float().t()).to(dtype)
        s["up"] = (s["x"].float() @ s["up_weight"].float().t()).to(dtype)
        s["dy"] = (0.02 * normal(rows, hidden)).to(dtype)
        s["dx"] = torch.empty_like(s["x"])
        s["dgate_weight"], s["dup_weight"] = torch.empty_like(s["gate_weight"]), torch.empty_like(s["up_weight"])
        return s
    vocab = case["vocab"]
    s["weight"] = (2 * width ** -0.5 * normal(vocab, width)).to(dtype)
    # frequent tokens first; half of the rows point towards their target's weight,
    # as a trained model's do
    u = torch.rand(rows, generator=g, device=dev)
    target = (torch.exp(u * math.log(vocab)).long() - 1).clamp(0, vocab - 1)
    known = (torch.rand((rows, 1), generator=g, device=dev) < 0.5).float()
    s["x"] = (x + 2.0 * known * s["weight"][target].float()).to(dtype)
    ignored = torch.rand(rows, generator=g, device=dev) < case["ignored"]
    s["target"] = torch.where(ignored, torch.full_like(target, IGNORE), target)
    if case["op"] == "loss":
        s["loss"], s["lse"] = (torch.empty(rows, device=dev) for _ in range(2))
        return s
    s["lse"] = torch.logsumexp(s["x"].float() @ s["weight"].float().t(), dim=1)
    counted = (~ignored).float()
    # the mean over the counted rows; in fp16 scaled up, as such a training's loss is
    s["dloss"] = counted * ((1024.0 if case["dtype"] == "fp16" else 1.0) / counted.sum().clamp_min(1.0))
    s["dx"], s["dweight"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
    return s


def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    if name == "gelu":
        cdf = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "gated":
        x = s["x"].float()
        g, u = x @ s["gate_weight"].float().t(), x @ s["up_weight"].float().t()
        y = (_act(case["act"], g)[0] * u).to(s["y"].dtype)
        if case["keep"]:
            return {"y": y, "gate": g.to(y.dtype), "up": u.to(y.dtype)}
        return {"y": y}
    if case["op"] == "gated_grad":
        x, dy, u = s["x"].float(), s["dy"].float(), s["up"].float()
        act, slope = _act(case["act"], s["gate"].float())
        dg, du = dy * u * slope, dy * act
        return {"dx": (dg @ s["gate_weight"].float() + du @ s["up_weight"].float()).to(s["dx"].dtype),
                "dgate_weight": (dg.t() @ x).to(s["dx"].dtype), "dup_weight": (du.t() @ x).to(s["dx"].dtype)}
    counted = s["target"] != IGNORE
    at = torch.where(counted, s["target"], torch.zeros_like(s["target"]))[:, None]
    logits = s["x"].float() @ s["weight"].float().t()
    if case["op"] == "loss":
        top = logits.amax(dim=1, keepdim=True)
        lse = (top + torch.log(torch.exp(logits - top).sum(dim=1, keepdim=True)))
        loss = torch.where(counted[:, None], lse - logits.gather(1, at), torch.zeros_like(lse))
        return {"loss": loss[:, 0], "lse": lse[:, 0]}
    dloss = torch.where(counted, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    dlogits = torch.exp(logits - s["lse"][:, None]) * dloss
    dlogits.scatter_add_(1, at, -dloss)
    x = torch.where(counted[:, None], s["x"], torch.zeros_like(s["x"])).float()
    return {"dx": (dlogits @ s["weight"].float()).to(s["dx"].dtype), "dweight": (dlogits.t() @ x).to(s["dweight"].dtype)}


def _own(s, case):
    import persistent_tile_scheduled_amd as tsg
    if case["op"] == "gated":
        tsg.gated_linear(s["x"], s["gate_weight"], s["up_weight"], s["y"], case["act"], gate=s.get("gate"), up=s.get("up"))
        return {name: s[name] for name in (("y", "gate", "up") if case["keep"] else ("y",))}
    if case["op"] == "gated_grad":
        tsg.gated_linear_grad(s["dy"], s["x"], s["gate_weight"], s["up_weight"], s["gate"], s["up"], s["dx"],
                              s["dgate_weight"], s["dup_weight"], case["act"])
        return {"dx": s["dx"], "dgate_weight": s["dgate_weight"], "dup_weight": s["dup_weight"]}
    if case["op"] == "loss":
        tsg.linear_cross_entropy(s["x"], s["weight"], s["target"], s["loss"], s["lse"], ignore_index=IGNORE)
        return {"loss": s["loss"], "lse": s["lse"]}
    tsg.linear_cross_entropy_grad(s["dloss"], s["x"], s["weight"], s["target"], s["lse"], s["dx"], s["dweight"], ignore_index=IGNORE)
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _exact_act(name, g):
    if name == "silu":
        p = torch.sigmoid(g)
        return p * g, p + g * p * torch.sigmoid(-g)
    if name == "gelu":
        p = torch.special.ndtr(g)
        return p * g, p + g * (g * g * -0.5).exp() / (2 * math.pi) ** 0.5
    # (1 + tanh z) / 2 is the logistic function of 2 z
    k = 2 * (2 / math.pi) ** 0.5
    p = torch.sigmoid(k * g * (1 + 0.044715 * g.square()))
    return p * g, p + g * p * (1 - p) * k * (1 + 0.134145 * g.square())


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "gated":
        g = torch.matmul(x, s["gate_weight"].double().t())
        u = torch.matmul(x, s["up_weight"].double().t())
        out = {"y": _exact_act(case["act"], g)[0] * u}
        return {**out, "gate": g, "up": u} if case["keep"] else out
    if case["op"] == "gated_grad":
        act, slope = _exact_act(case["act"], s["gate"].double())
        dy = s["dy"].double()
        du, dg = act * dy, slope * s["up"].double() * dy
        dx = torch.matmul(du, s["up_weight"].double())
        dx += torch.matmul(dg, s["gate_weight"].double())
        return {"dx": dx, "dgate_weight": torch.matmul(dg.t(), x), "dup_weight": torch.matmul(du.t(), x)}
    rows = torch.arange(x.shape[0], device=x.device)
    kept = s["target"].ne(IGNORE)
    logits = torch.matmul(x, s["weight"].double().t())
    if case["op"] == "loss":
        lse = torch.logsumexp(logits, dim=1)
        return {"loss": (lse - logits[rows, s["target"].clamp_min(0)]) * kept, "lse": lse}
    logits -= s["lse"].double()[:, None]
    logits.exp_()
    logits[rows[kept], s["target"][kept]] -= 1.0
    logits *= (s["dloss"].double() * kept)[:, None]
    return {"dx": torch.matmul(logits, s["weight"].double()), "dweight": torch.matmul(logits.t(), x)}
