"""Infinities and NaN in the routed-expert layer's rows: they reach what they
belong to and nothing else."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from tests.gpu_util import dev
from tests.moe_util import i32, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H", [9, 20, 515, 4099])
def test_combine_weight_gradient_with_an_infinite_column(H, dtype):
    """One infinite product in any column is an infinite dot, those among the columns that two chunks share included."""
    cols = sorted({0, 1, H // 2, *range(max(0, H - 16), H)})
    T = len(cols)
    plan = mxq.moe_plan(i32(np.arange(T)[:, None] % 4), 4)
    rows = plan.rows[:, 0].long()
    at = torch.tensor(cols, device=dev())
    go = torch.ones(T, H, device=dev()).to(values(np.random.default_rng(0), (1,), dtype).dtype)
    for bad in (float("inf"), float("-inf")):
        y = values(np.random.default_rng(H), (T, H), dtype)
        y[rows, at] = bad
        w = torch.ones(T, 1, device=dev(), requires_grad=True)
        gw, = torch.autograd.grad(mxq.moe_combine(y, w, plan), w, go)
        assert (gw == bad).all(), (gw[:, 0].tolist(), cols)
        y = values(np.random.default_rng(H), (T, H), dtype).abs() + 1      # an infinite gradient, finite rows
        g = go.clone()
        g[torch.arange(T, device=dev()), at] = bad
        gw, = torch.autograd.grad(mxq.moe_combine(y, w, plan), w, g)
        assert (gw == bad).all(), (gw[:, 0].tolist(), cols)
