"""A normalised linear layer trained with block-scaled FP8 activations: how
layer_norm, mx_quantize, run_mx, mx_weight_grad, mx_dequantize, Plan.run and
layer_norm_grad go together.

    layer = MxNormLinear(width=4096, out=8192)
    y, saved = layer.forward(x)              # x [rows, width], y [rows, out], bfloat16
    dx, grads = layer.backward(dy, saved)    # grads: gamma, beta, weight in float32

Forward: the normalised rows leave layer_norm as MX and are both the product's
operand and what is kept for the backward pass (33/32 bytes a value; the
normalised activation is never written in 16 bits).  Backward: the weight's
gradient comes straight from those codes, the input's from the weight as the
forward product saw it, read back from its codes.

    python -m persistent_tile_scheduled_amd.mx_linear     # three training steps on cuda:0
"""

from __future__ import annotations

import torch

from . import Plan, layer_norm, layer_norm_grad, mx_dequantize, mx_quantize, mx_weight_grad


class MxNormLinear:
    """y = layer_norm(x) @ weight^T with bfloat16 activations; float32 master
    parameters gamma[width], beta[width] and weight[out, width]."""

    def __init__(self, width: int, out: int, eps: float = 1e-5, device="cuda", seed: int = 0):
        if width % 128 or out % 64:
            raise ValueError("width must be divisible by 128 and out by 64 (the products' slabs)")
        g = torch.Generator().manual_seed(seed)
        self.width, self.out, self.eps = width, out, eps
        self.gamma = torch.ones(width, device=device)
        self.beta = torch.zeros(width, device=device)
        self.weight = (torch.randn((out, width), generator=g) / width ** 0.5).to(device)

    @staticmethod
    def _held(rows, width, device):
        return (torch.empty((rows, width), dtype=torch.float8_e4m3fn, device=device),
                torch.empty((rows, width // 32), dtype=torch.float8_e8m0fnu, device=device))

    def forward(self, x):
        rows, dev = x.shape[0], x.device
        codes, scales = self._held(rows, self.width, dev)
        wcodes, wscales = self._held(self.out, self.width, dev)
        mean, rstd = (torch.empty(rows, device=dev) for _ in range(2))
        layer_norm(x, self.gamma, self.beta, self.eps, mean=mean, rstd=rstd, codes=codes, scales=scales)
        mx_quantize(self.weight, wcodes, wscales)
        y = torch.empty((rows, self.out), dtype=torch.bfloat16, device=dev)
        Plan(rows, self.out, self.width, "mxfp8", 256, 256, 128, 8, 2).run_mx(codes, scales, wcodes, wscales, y)
        return y, (x, mean, rstd, codes, scales, wcodes, wscales)

    def backward(self, dy, saved):
        x, mean, rstd, codes, scales, wcodes, wscales = saved
        rows, dev = x.shape[0], x.device
        grads = {"gamma": torch.empty_like(self.gamma), "beta": torch.empty_like(self.beta),
                 "weight": torch.empty_like(self.weight)}
        mx_weight_grad(dy, codes, scales, grads["weight"])
        weight = torch.empty((self.out, self.width), dtype=torch.bfloat16, device=dev)
        mx_dequantize(wcodes, wscales, weight)
        dn = torch.empty((rows, self.width), dtype=torch.bfloat16, device=dev)
        Plan(rows, self.width, self.out, "bf16", 256, 256, 64, 8, 3).run(dy, weight, dn)
        dx = torch.empty_like(x)
        layer_norm_grad(dn, x, self.gamma, mean, rstd, dx, grads["gamma"], grads["beta"])
        return dx, grads


def train(steps: int = 3, rows: int = 4096, width: int = 1024, out: int = 2048, device="cuda"):
    """Fits a layer to random targets by gradient descent, losses step by step.
    The step sizes are below 2 over the largest curvature of the mean square: that
    of the weight is (2 / out) times the largest eigenvalue of the rows' second
    moments, about (1 + (width / rows)^(1/2))^2 (here 1 / 450); those of gamma and
    beta are two to three times it."""
    layer = MxNormLinear(width, out, device=device)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((rows, width), generator=g).to(device).bfloat16()
    target = torch.randn((rows, out), generator=g).to(device)
    losses = []
    for _ in range(steps):
        y, saved = layer.forward(x)
        diff = y.float() - target
        dx, grads = layer.backward((diff * (2.0 / diff.numel())).bfloat16(), saved)
        for name, grad in grads.items():
            getattr(layer, name).sub_(grad, alpha=4e2 if name == "weight" else 1e2)
        losses.append(diff.square().mean().item())
    return losses


if __name__ == "__main__":
    for step, loss in enumerate(train()):
        print(f"step {step}: loss {loss:.5f}")
