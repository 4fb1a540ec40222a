"""Layer norm's gradient for rows wider than one launch may have threads over 32."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg

pytestmark = pytest.mark.gpu


def test_columns_past_a_launch():
    """2^27 + 40 columns of two rows with mean 0 and rstd 1: every product of two bf16 is exact in fp32, so
    dgamma and dbeta are one fp32 addition each."""
    dev, width = torch.device("cuda:0"), (1 << 27) + 40
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x, dy = (torch.randn((2, width), generator=g, device=dev).bfloat16() for _ in range(2))
    mean, rstd = torch.zeros(2, device=dev), torch.ones(2, device=dev)
    dx, dgamma, dbeta = torch.empty_like(x), *(torch.full((width,), float("nan"), device=dev) for _ in range(2))
    tsg.layer_norm_grad(dy, x, None, mean, rstd, dx, dgamma, dbeta)
    assert torch.equal(dbeta, dy[0].float() + dy[1].float())
    assert torch.equal(dgamma, dy[0].float() * x[0].float() + dy[1].float() * x[1].float())
