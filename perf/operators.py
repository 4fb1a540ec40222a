"""What is measured of the operators around the block-scaled FP8 product when a
normalised linear layer is trained: layer norm and its gradient, activations
held in 8 bits (MX: E4M3 codes, one E8M0 scale per 32 along the row) and read
back, and the weight's gradient from the 8-bit activation.

A case is one call.  `run` makes it either through the library (`own`) or in
its plain form: elementary torch operations in fp32, rounded once at the end.
`exact` gives the same outputs from the definitions in fp64.
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}
EPS = 1e-5
MOST_VALUES = 8192 * 8192        # of one activation
MOST_PRODUCTS = 8192 ** 3        # of one weight gradient


def listed():
    return [
        # one token's hidden state on its way through a decoder: latency
        {"name": "norm one row bf16", "op": "norm", "rows": 1, "width": 4096, "dtype": "bf16", "weights": "bf16", "codes": False},
        # a ragged batch (rows and width that no tile divides), fp32 master weights
        {"name": "norm ragged fp16", "op": "norm", "rows": 16000, "width": 4000, "dtype": "fp16", "weights": "fp32", "codes": False},
        # a training batch normalised straight into the product's operand and checkpoint
        {"name": "norm to codes bf16", "op": "norm", "rows": 8192, "width": 8192, "dtype": "bf16", "weights": "bf16", "codes": True},
        # a small model's backward pass: latency, and the column sums' tail
        {"name": "norm grad small fp16", "op": "norm_grad", "rows": 512, "width": 512, "dtype": "fp16", "weights": "fp16"},
        # a training batch's backward pass
        {"name": "norm grad large bf16", "op": "norm_grad", "rows": 8192, "width": 8192, "dtype": "bf16", "weights": "fp32"},
        # a small activation checkpoint
        {"name": "quantize small fp16", "op": "quantize", "rows": 512, "width": 512, "dtype": "fp16"},
        # a training batch's checkpoint
        {"name": "quantize large bf16", "op": "quantize", "rows": 16384, "width": 4096, "dtype": "bf16"},
        # the same two read back for a backward pass that wants ordinary values
        {"name": "dequantize small fp16", "op": "dequantize", "rows": 1024, "width": 1024, "dtype": "fp16"},
        {"name": "dequantize large bf16", "op": "dequantize", "rows": 8192, "width": 8192, "dtype": "bf16"},
        # a small layer: fewer output tiles than compute units
        {"name": "weight grad small fp16", "op": "weight_grad", "rows": 512, "out": 512, "width": 512, "dtype": "fp16", "grad": "fp16"},
        # a narrow layer over a long batch: few output tiles, a long sum; fp32 master gradients
        {"name": "weight grad long bf16", "op": "weight_grad", "rows": 32768, "out": 2048, "width": 2048, "dtype": "bf16", "grad": "fp32"},
        # a wide layer
        {"name": "weight grad large bf16", "op": "weight_grad", "rows": 8192, "out": 8192, "width": 8192, "dtype": "bf16", "grad": "bf16"},
    ]


def draw(rng):
    def size(low, high, step=1):
        v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        return max(low, min(high, v // step * step))

    op = rng.choice(("norm", "norm_grad", "quantize", "dequantize", "weight_grad"))
    half = rng.choice(("fp16", "bf16"))
    if op == "weight_grad":
        out, width = size(64, 8192, 8), size(64, 8192, 32)
        rows = size(1, min(65536, MOST_PRODUCTS // (out * width)))
        return {"op": op, "rows": rows, "out": out, "width": width, "dtype": half, "grad": rng.choice((half, "fp32"))}
    codes = op in ("quantize", "dequantize") or (op == "norm" and rng.random() < 0.5)
    width = size(64, 16384, 32 if codes else rng.choice((1, 2, 8, 64)))
    case = {"op": op, "rows": size(1, min(65536, MOST_VALUES // width)), "width": width,
            "dtype": rng.choice((half, half, "fp32"))}
    if case["dtype"] == "fp32":
        case["rows"] = max(1, case["rows"] // 2)
    if op in ("norm", "norm_grad"):
        case["weights"] = rng.choice((case["dtype"], "fp32"))
    if op == "norm":
        case["codes"] = codes
    return case


def work(case):
    rows, width, e = case["rows"], case["width"], BYTES[case["dtype"]]
    values, held = rows * width, rows * width + rows * (width // 32)
    if case["op"] == "norm":
        w = BYTES[case["weights"]]
        return {"bytes": values * e + (held if case["codes"] else values * e) + 2 * width * w + 8 * rows, "flops": 8 * values}
    if case["op"] == "norm_grad":
        w = BYTES[case["weights"]]
        return {"bytes": 3 * values * e + 3 * width * w + 8 * rows, "flops": 13 * values}
    if case["op"] in ("quantize", "dequantize"):
        return {"bytes": values * e + held, "flops": 3 * values}
    out = case["out"]
    return {"bytes": held + rows * out * e + out * width * BYTES[case["grad"]], "flops": 2 * rows * out * width}


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows, width, dtype = case["rows"], case["width"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # hidden states: channels of different size, a few of them far larger, rows of
    # different size, and a mean that is not zero
    spread = torch.exp(0.5 * normal(width))
    spread = torch.where(torch.rand(width, generator=g, device=dev) < 0.01, 10 * spread, spread)
    x = (normal(rows, width) * spread * torch.exp(0.3 * normal(rows, 1)) + 0.25).to(dtype)
    s = {"case": dict(case)}
    if case["op"] in ("norm", "norm_grad"):
        weights = DTYPES[case["weights"]]
        s["x"], s["gamma"] = x, (1 + 0.1 * normal(width)).to(weights)
        s["beta"] = (0.1 * normal(width)).to(weights)
        s["mean"] = torch.empty(rows, device=dev)
        s["rstd"] = torch.empty(rows, device=dev)
        if case["op"] == "norm_grad":
            s["dy"] = (0.02 * normal(rows, width)).to(dtype)
            s["mean"], s["rstd"] = (t.float() for t in _moments(x.double()))
            s["dx"] = torch.empty_like(x)
            s["dgamma"], s["dbeta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["beta"])
        elif case["codes"]:
            s["codes"], s["scales"] = _held(rows, width, dev)
        else:
            s["y"] = torch.empty_like(x)
    elif case["op"] == "quantize":
        s["x"] = x
        s["codes"], s["scales"] = _held(rows, width, dev)
    else:
        s["codes"], s["scales"] = _encode(x.float())
        if case["op"] == "dequantize":
            s["out"] = torch.empty_like(x)
        else:
            s["dy"] = (0.02 * normal(rows, case["out"])).to(dtype)
            s["dw"] = torch.empty((case["out"], width), dtype=DTYPES[case["grad"]], device=dev)
    return s


def _held(rows, width, dev):
    return (torch.empty((rows, width), dtype=torch.float8_e4m3fn, device=dev),
            torch.empty((rows, width // 32), dtype=torch.float8_e8m0fnu, device=dev))


def _moments(x):
    mean = x.mean(dim=1)
    return mean, torch.rsqrt((x - mean[:, None]).square().mean(dim=1) + EPS)


def _encode(v):
    """fp32 rows -> E4M3 codes and E8M0 scales: the largest magnitude of a block
    of 32 gets E4M3's largest exponent, 8; what is past 448 is held as 448."""
    blocks = v.view(v.shape[0], -1, 32)
    _, exponent = torch.frexp(blocks.abs().amax(dim=2))
    shared = (exponent - 9).clamp(-127, 127)
    shared = torch.where(blocks.abs().amax(dim=2) > 0, shared, torch.full_like(shared, -127))
    scaled = torch.ldexp(blocks, -shared[:, :, None]).clamp(-448.0, 448.0)
    return (scaled.to(torch.float8_e4m3fn).view(v.shape),
            (shared + 127).to(torch.uint8).view(torch.float8_e8m0fnu))


def _decode(codes, scales):
    return (codes.float().view(codes.shape[0], -1, 32) * scales.float()[:, :, None]).view(codes.shape)


def run(s):
    case = s["case"]
    if own:
        return _own(s, case["op"])
    if case["op"] == "norm":
        x = s["x"].float()
        mean, rstd = _moments(x)
        y = (x - mean[:, None]) * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        if case["codes"]:
            codes, scales = _encode(y)
            return {"codes": codes, "scales": scales, "mean": mean, "rstd": rstd}
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if case["op"] == "norm_grad":
        dy = s["dy"].float()
        normed = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["gamma"].float()
        dx = (g - g.mean(dim=1, keepdim=True) - normed * (g * normed).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
        return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * normed).sum(dim=0).to(s["gamma"].dtype),
                "dbeta": dy.sum(dim=0).to(s["gamma"].dtype)}
    if case["op"] == "quantize":
        codes, scales = _encode(s["x"].float())
        return {"codes": codes, "scales": scales}
    if case["op"] == "dequantize":
        return {"out": _decode(s["codes"], s["scales"]).to(s["out"].dtype)}
    return {"dw": (s["dy"].float().t() @ _decode(s["codes"], s["scales"])).to(s["dw"].dtype)}


def _own(s, op):
    import persistent_tile_scheduled_amd as tsg
    if op == "norm":
        if "codes" in s:
            tsg.layer_norm(s["x"], s["gamma"], s["beta"], EPS, mean=s["mean"], rstd=s["rstd"], codes=s["codes"], scales=s["scales"])
            return {"codes": s["codes"], "scales": s["scales"], "mean": s["mean"], "rstd": s["rstd"]}
        tsg.layer_norm(s["x"], s["gamma"], s["beta"], EPS, y=s["y"], mean=s["mean"], rstd=s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_grad":
        tsg.layer_norm_grad(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "quantize":
        tsg.mx_quantize(s["x"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "dequantize":
        tsg.mx_dequantize(s["codes"], s["scales"], s["out"])
        return {"out": s["out"]}
    tsg.mx_weight_grad(s["dy"], s["codes"], s["scales"], s["dw"])
    return {"dw": s["dw"]}


def _exact_codes(v):
    """Codes' and scales' values in fp64: the scale from the binary exponent of
    the block's largest magnitude, the code by rounding to E4M3's grid (four
    significant bits, steps of 2^-9 below 2^-6), ties to even."""
    rows, width = v.shape
    b = v.reshape(rows, width // 32, 32)
    top = b.abs().max(dim=2).values
    power = torch.floor(torch.log2(top.clamp_min(2.0 ** -140)))
    power = power + (torch.exp2(power + 1) <= top).double() - (torch.exp2(power) > top).double()
    scale = torch.exp2((power - 8).clamp(-127.0, 127.0))
    q = b / scale[:, :, None]
    del b
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    q = (torch.round(q / step) * step).clamp(-448.0, 448.0)
    return q.reshape(rows, width), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        mean = x.sum(dim=1) / x.shape[1]
        x -= mean[:, None]
        rstd = (x.square().sum(dim=1) / x.shape[1] + EPS).pow(-0.5)
        x *= rstd[:, None]
        x *= s["gamma"].double()
        x += s["beta"].double()
        if case["codes"]:
            codes, scales = _exact_codes(x)
            return {"codes": codes, "scales": scales, "mean": mean, "rstd": rstd}
        return {"y": x, "mean": mean, "rstd": rstd}
    if case["op"] == "norm_grad":
        n = s["x"].shape[1]
        h = (s["x"].double() - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
        dy = s["dy"].double()
        dgamma, dbeta = (dy * h).sum(dim=0), dy.sum(dim=0)
        dy *= s["gamma"].double()
        along, across = (dy * h).sum(dim=1) / n, dy.sum(dim=1) / n
        dy -= across[:, None] + h * along[:, None]
        dy *= s["rstd"].double()[:, None]
        return {"dx": dy, "dgamma": dgamma, "dbeta": dbeta}
    if case["op"] == "quantize":
        codes, scales = _exact_codes(s["x"].double())
        return {"codes": codes, "scales": scales}
    scale = s["scales"].view(torch.uint8).double() - 127
    value = s["codes"].double() * torch.exp2(scale).repeat_interleave(32, dim=1)
    if case["op"] == "dequantize":
        return {"out": value}
    return {"dw": torch.matmul(s["dy"].double().t(), value)}
