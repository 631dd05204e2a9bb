"""Infinities and NaN in the routed-expert layer's rows: they reach what they
belong to and nothing else, and finite rows make none."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from oracle import moe
from tests.gpu_util import dev
from tests.moe_util import assert_rounded, f64, i32, values
from tests.test_gpu_swiglu import bound_grad

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


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("checkpoint", ["fp8", None])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_swiglu_overflow_reaches_the_gradients(dtype, checkpoint, bad):
    """An inf or a NaN in gate or up is one in h and in the gradients at its place, kept in 8 bits or whole (what a loss
    scaler looks for); other rows, and other blocks of 32 columns, are as without it."""
    I, R = 96, 40
    g = np.random.default_rng(1)
    x = values(g, (R, 2 * I), dtype)
    gh = values(g, (R, I), dtype)
    hit = x.clone()
    cols = g.integers(0, I, R)
    up = np.arange(R) % 2 == 1
    put = torch.from_numpy(cols + np.where(up, I, 0)).to(dev())
    rows = torch.arange(0, R - 4, device=dev())                        # the last four rows stay as they are
    hit[rows, put[rows]] = bad
    res = []
    for t in (x, hit):
        leaf = t.clone().requires_grad_(True)
        h = mxq.swiglu(leaf, checkpoint=checkpoint)
        res.append((h.detach(), torch.autograd.grad(h, leaf, gh)[0]))
    (h0, g0), (h1, g1) = res
    at = torch.from_numpy(cols).to(dev())[rows]
    assert not torch.isfinite(h1[rows, at]).any()
    assert not torch.isfinite(g1[rows, at]).any()                      # gate's gradient takes both factors
    gate = torch.from_numpy(~up).to(dev())[rows]
    assert not torch.isfinite(g1[rows, at + I])[gate].any()            # up's gradient is a multiple of silu(gate)
    block = torch.zeros(R, I, dtype=torch.bool, device=dev())
    block.view(R, -1, 32)[rows, at // 32] = True
    assert torch.equal(h0[~block], h1[~block])
    both = torch.cat([block, block], 1)
    assert torch.equal(g0[~both], g1[~both]) and torch.isfinite(g0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_carry_infinities_and_nan(dtype):
    """Dispatch copies them; combine and the dispatch's gradient pass them on to their token and column alone."""
    g = np.random.default_rng(2)
    T, k, H = 6, 2, 21
    plan = mxq.moe_plan(i32(g.integers(0, 3, (T, k))), 3)
    x = values(g, (T, H), dtype)
    x[1, 15], x[2, 20], x[3, 0] = float("inf"), float("nan"), float("-inf")
    out = mxq.moe_dispatch(x, plan)
    assert torch.equal(torch.nan_to_num(out, 7.0), torch.nan_to_num(x[plan.slots.long() // k], 7.0))
    w = torch.full((T, k), 0.5, device=dev())
    back = mxq.moe_combine(out, w, plan)
    assert torch.equal(torch.isfinite(back), torch.isfinite(x)) and back[1, 15] == float("inf") and back[2, 20].isnan()
    leaf = values(g, (T, H), dtype).requires_grad_(True)
    gx, = torch.autograd.grad(mxq.moe_dispatch(leaf, plan), leaf, out)
    assert torch.equal(torch.isfinite(gx), torch.isfinite(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("checkpoint", ["fp8", None])
def test_swiglu_gradients_of_far_values_stay_finite(dtype, checkpoint):
    """A gate far below 0 has a sigmoid of 0: no product of the others is large enough to make its gradients NaN."""
    far = [-1e38, -2e38, -1e30, -1e20, -200.0, 200.0, 1e20, 1e30]
    size = [1.0, -1e12, 1e30, -3e37]
    R, I = len(far) * len(size), 32
    x, gh = values(np.random.default_rng(3), (R, 2 * I), dtype), values(np.random.default_rng(4), (R, I), dtype)
    for r in range(R):
        gate, d = far[r % len(far)], size[r // len(far)]
        x[r, :I] = gate
        x[r, I::2] *= 1e30 if gate < 0 else 1.0
        gh[r] = (gh[r].float().clamp(-2, 2) * (d if gate < 0 else 1e-3)).to(gh.dtype)
    leaf = x.clone().requires_grad_(True)
    grad, = torch.autograd.grad(mxq.swiglu(leaf, checkpoint=checkpoint), leaf, gh)
    at = f64(x) if checkpoint is None else moe.kept(f64(x))
    want = moe.swiglu_grad(at, f64(gh))
    assert np.isfinite(want).all() and torch.isfinite(grad).all()
    for r in range(R):                                       # each row on its own: a bound takes the largest values it sees
        one = slice(r, r + 1)
        assert_rounded(grad[one], want[one], dtype, bound_grad(at[one], f64(gh)[one]), "grad")
