"""Up to 32 rows in either kernel, for few rows or of tiles, by what the rule gives them."""

import pytest
import torch

import persistent_tile_scheduled_amd as tsg
from tests.linear_cases import BF16, DEV, FP16, check_gated, check_loss, gated_inputs, loss_inputs
from tests.linear_rule import FEW, TILE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weights,rows,width,columns", FEW + TILE)
@pytest.mark.parametrize("dtype", [FP16, BF16], ids=str)
def test_few_rows(dtype, weights, rows, width, columns):
    if weights == 2:
        x, wg, wu = gated_inputs(rows, width, columns, dtype, 61)
        y, gate, up = (torch.full((rows, columns), float("nan"), dtype=dtype, device=DEV) for _ in range(3))
        tsg.gated_linear(x, wg, wu, y, "silu", gate=gate, up=up)
        check_gated(x, wg, wu, "silu", y, gate, up, "few rows")
    else:
        x, w, target = loss_inputs(rows, width, columns, dtype, 62)
        loss, lse = (torch.full((rows,), float("nan"), device=DEV) for _ in range(2))
        tsg.linear_cross_entropy(x, w, target, loss, lse)
        check_loss(x, w, target, loss, lse, "few rows")
