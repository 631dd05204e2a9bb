"""GPU parity of the grouped order (moe_plan), dispatch (plain and quantized)
and combine, with their gradients, against the float64 oracle."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from nvfp4_quantization_grouped_amd import _lib
from oracle import moe
from tests.gpu_util import DTYPES, dev
from tests.moe_util import U, assert_rounded, f64, i32, values

pytestmark = pytest.mark.gpu


def random_experts(g, T, k, E, drop=0.1):
    e = g.integers(0, E, (T, k))
    e[g.random((T, k)) < drop] = -1
    return e.astype(np.int32)


def check_plan(e, E, first, local):
    plan = mxq.moe_plan(i32(e), E, first, local)
    flat = e.reshape(-1).astype(np.int64) - first
    key = np.where((flat >= 0) & (flat < local), flat, local)
    slots = np.argsort(key, kind="stable")
    offs = np.cumsum(np.bincount(key, minlength=local + 1)[:local])
    rows = np.empty_like(slots)
    rows[slots] = np.arange(slots.size)
    rows = np.where(key < local, rows, ~rows)
    assert np.array_equal(plan.offs.cpu().numpy(), offs), "offs"
    assert np.array_equal(plan.slots.cpu().numpy(), slots), "slots"
    assert np.array_equal(plan.rows.cpu().numpy().reshape(-1), rows), "rows"
    return plan


@pytest.mark.parametrize("T,k,E,first,local", [
    (1, 1, 1, 0, 1), (1, 8, 256, 0, 256), (7, 3, 5, 0, 5), (64, 8, 32, 8, 16), (1000, 6, 60, 0, 60), (2048, 8, 256, 0, 256),
    (16384, 1, 8, 0, 8), (2049, 8, 256, 0, 256), (4099, 7, 64, 32, 32), (65536, 8, 256, 0, 256), (3000, 8, 1024, 0, 1024),
    (1500, 12, 1024, 0, 1024), (33333, 1, 3, 1, 2), (20000, 2, 1024, 1000, 24), (131072, 9, 128, 0, 128), (0, 8, 16, 0, 16)])
def test_plan(T, k, E, first, local):
    """One workgroup and many, one expert and 1024, slots of experts elsewhere."""
    check_plan(random_experts(np.random.default_rng(T + k + E), T, k, E), E, first, local)


def test_plan_extremes():
    g = np.random.default_rng(1)
    for T, k in ((50, 4), (9000, 4)):
        for e in (np.zeros((T, k)), np.full((T, k), -1), np.full((T, k), 31),                 # all in one place, or none
                  g.choice([-2 ** 31, -5, 0, 31, 32, 1000, 2 ** 31 - 1], (T, k))):
            check_plan(e.astype(np.int32), 32, 0, 32)
    # the oracle's own slot-by-slot order
    e = random_experts(g, 40, 5, 9)
    plan = check_plan(e, 9, 2, 5)
    for got, want in zip(plan, moe.plan(e, 2, 5)):
        assert np.array_equal(got.cpu().numpy(), want)
    # an index that is a view with strides
    wide = i32(random_experts(g, 100, 16, 20))
    a, b = mxq.moe_plan(wide[:, 3:9], 20), mxq.moe_plan(wide[:, 3:9].clone(), 20)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_plan_refusals():
    e = torch.zeros(4, 2, dtype=torch.int32, device=dev())
    with pytest.raises(TypeError):
        mxq.moe_plan(e.long(), 4)
    with pytest.raises(ValueError):
        mxq.moe_plan(e.view(-1), 4)
    for kw in (dict(num_experts=4, first_expert=-1), dict(num_experts=4, first_expert=2, local_experts=3),
               dict(num_experts=0), dict(num_experts=2000)):
        with pytest.raises(ValueError):
            mxq.moe_plan(e, **kw)


SHAPES = [(1, 8, 1, 4), (5, 256, 3, 8), (16, 7168, 8, 256), (33, 100, 4, 8), (9, 7, 2, 3), (6, 1, 5, 4), (130, 2056, 6, 16),
          (3, 20000, 2, 4), (257, 33, 8, 32), (2, 4099, 33, 40), (40, 512, 1, 8)]


@pytest.mark.parametrize("T,H,k,E", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_dispatch(T, H, k, E, dtype):
    g = np.random.default_rng(T * H + k)
    e = random_experts(g, T, k, E)
    first = E // 4
    plan = mxq.moe_plan(i32(e), E, first, E - first)
    rows = plan.rows.cpu().numpy()
    x = values(g, (T, H), dtype).requires_grad_(True)
    out = mxq.moe_dispatch(x, plan)
    want = moe.dispatch(f64(x), rows)
    assert np.array_equal(f64(out), want) and out.dtype == x.dtype
    assert torch.equal(out, mxq.moe_dispatch(x.detach(), plan))
    go = values(g, (T * k, H), dtype)
    go[int(plan.offs[-1]):] = float("nan")                # rows behind the last expert are not read
    gx, = torch.autograd.grad(out, x, go)
    gs = f64(go)
    # k fp32 additions of the absolute values
    total = moe.dispatch_grad(np.abs(np.nan_to_num(gs)), rows)
    assert_rounded(gx, moe.dispatch_grad(np.nan_to_num(gs), rows), dtype, k * U * total, "grad_x")


@pytest.mark.parametrize("T,H,k,E", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_combine(T, H, k, E, dtype):
    g = np.random.default_rng(T * H + k + 1)
    e = random_experts(g, T, k, E)
    first = E // 4
    plan = mxq.moe_plan(i32(e), E, first, E - first)
    rows = plan.rows.cpu().numpy()
    y = values(g, (T * k, H), dtype)
    y[int(plan.offs[-1]):] = float("nan")                 # what no expert wrote is not read
    w = values(g, (T, k), "f32")
    w[plan.rows < 0] = float("nan")                       # nor are the weights of slots that are not served
    y.requires_grad_(True)
    w.requires_grad_(True)
    out = mxq.moe_combine(y, w, plan)
    ys, ws = np.nan_to_num(f64(y)), np.nan_to_num(f64(w))
    assert_rounded(out, moe.combine(ys, ws, rows), dtype, (k + 1) * U * moe.combine(np.abs(ys), np.abs(ws), rows), "out")
    go = values(g, (T, H), dtype)
    gy, gw = torch.autograd.grad(out, (y, w), go, retain_graph=True)
    want_y, want_w = moe.combine_grad(f64(go), ys, ws, rows)
    _, abs_w = moe.combine_grad(np.abs(f64(go)), np.abs(ys), ws, rows)
    assert_rounded(gy, want_y, dtype, U * np.abs(want_y), "grad_y")
    # a lane adds at most H / 64 products, lanes and waves meet in 16 additions at most
    assert_rounded(gw, want_w, "f32", (H / 64 + 24) * U * abs_w, "grad_weights")
    # one gradient alone is the same
    assert torch.equal(torch.autograd.grad(mxq.moe_combine(y, w.detach(), plan), y, go)[0], gy)
    assert torch.equal(torch.autograd.grad(mxq.moe_combine(y.detach(), w, plan), w, go)[0], gw)


@pytest.mark.parametrize("T,H,k", [(1, 32, 1), (5, 96, 3), (64, 7168, 8), (33, 2048, 6), (9, 512, 33), (3, 32 * 257, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("format", ["fp8", "mxfp4"])
def test_dispatch_quantized(T, H, k, dtype, format):
    """Bit for bit what quantizing the dispatched rows gives."""
    g = np.random.default_rng(T + H)
    x = values(g, (T, H), dtype) * torch.exp2(torch.from_numpy(g.integers(-20, 5, (T, 1))).float()).to(dev()).to(DTYPES[dtype])
    x[0, :32] = 0.0
    x[0, 0] = -0.0
    x[T // 2] = x[T // 2] * 1e-6
    plan = mxq.moe_plan(i32(random_experts(g, T, k, 8, 0.3)), 8, 2, 5)
    codes, scales = mxq.moe_dispatch_quantized(x, plan, format)
    rows = mxq.moe_dispatch(x, plan)
    want = mxq.quantize_cache_packed(rows, "fp8", 32) if format == "fp8" else mxq.quantize_mxfp4(rows)
    assert codes.dtype == want[0].dtype and scales.dtype == want[1].dtype
    assert torch.equal(codes, want[0]) and torch.equal(scales.view(torch.uint8), want[1].view(torch.uint8))


def test_rows_strides_alignment_and_empty():
    g = np.random.default_rng(3)
    e = i32(random_experts(g, 20, 4, 8))
    plan = mxq.moe_plan(e, 8)
    for dtype in ("bf16", "f32"):
        base = values(g, (20, 2 * 101), dtype)
        for x in (base[:, 1:102], base[:, ::2], base.view(-1)[1:20 * 101 + 1].view(20, 101)):
            assert torch.equal(mxq.moe_dispatch(x, plan), mxq.moe_dispatch(x.clone(), plan))
        y = values(g, (80, 101), dtype).t().contiguous().t()
        w = values(g, (4, 20), "f32").t()
        assert torch.equal(mxq.moe_combine(y, w, plan), mxq.moe_combine(y.contiguous(), w.contiguous(), plan))
        # a broadcast gradient (stride 0)
        leaf = y.contiguous().requires_grad_(True)
        wl = w.contiguous().requires_grad_(True)
        a = torch.autograd.grad(mxq.moe_combine(leaf, wl, plan).sum(), (leaf, wl))
        b = torch.autograd.grad(mxq.moe_combine(leaf, wl, plan), (leaf, wl), torch.ones(20, 101, device=dev(), dtype=y.dtype))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    empty = mxq.moe_plan(e[:0], 8)
    assert empty.offs.tolist() == [0] * 8
    x = torch.zeros(0, 64, device=dev(), requires_grad=True)
    out = mxq.moe_dispatch(x, empty)
    assert out.shape == (0, 64) and torch.autograd.grad(out.sum(), x)[0].shape == (0, 64)
    nothing = mxq.moe_dispatch(torch.zeros(20, 0, device=dev()), plan)
    wl = torch.ones(20, 4, device=dev(), requires_grad=True)
    out = mxq.moe_combine(nothing, wl, plan)
    assert out.shape == (20, 0) and (torch.autograd.grad(out.sum(), wl)[0] == 0).all()


def test_rows_out_of_range_touch_nothing():
    """Row values that name no row: nothing is read or written for them (entry points called directly, the buffers
    inside larger ones with guards on both sides)."""
    g = np.random.default_rng(4)
    T, k, H = 3, 2, 40
    n = T * k
    bad = np.array([[0, n], [2 ** 31 - 1, 1], [-(n + 1), ~2]], np.int32)      # two rows served, one zeroed
    rows, L, s = i32(bad), _lib.moe_lib(), torch.cuda.current_stream().cuda_stream
    x = values(g, (T, H), "f32")
    pad = torch.full((n + 2, H), 5.0, device=dev())
    assert L.moe_dispatch(x.data_ptr(), 0, T, H, k, rows.data_ptr(), pad[1:].data_ptr(), s) == 0
    want = torch.full((n + 2, H), 5.0, device=dev())
    want[1], want[2], want[3] = x[0], x[1], 0.0
    assert torch.equal(pad, want)
    y, w = values(g, (n, H), "f32"), values(g, (T, k), "f32")
    out = torch.empty(T, H, device=dev())
    assert L.moe_combine(y.data_ptr(), 0, T, H, k, rows.data_ptr(), w.data_ptr(), out.data_ptr(), s) == 0
    assert torch.equal(out, torch.stack([w[0, 0] * y[0], w[1, 1] * y[1], torch.zeros(H, device=dev())]))
    gy, gw = torch.full((n + 2, H), 5.0, device=dev()), torch.full((T, k), 5.0, device=dev())
    assert L.moe_combine_bwd(x.data_ptr(), y.data_ptr(), 0, T, H, k, rows.data_ptr(), w.data_ptr(), gy[1:].data_ptr(),
                             gw.data_ptr(), s) == 0
    want = torch.full((n + 2, H), 5.0, device=dev())
    want[1], want[2], want[3] = w[0, 0] * x[0], w[1, 1] * x[1], 0.0
    assert torch.equal(gy, want)
    assert gw[0, 1] == 0 and gw[1, 0] == 0 and (gw[2] == 0).all() and gw[0, 0] != 0
    codes, scales = torch.full((n + 2, 32), 5, dtype=torch.uint8, device=dev()), torch.full((n + 2, 1), 5, dtype=torch.uint8, device=dev())
    x32 = x[:, :32].contiguous()
    assert L.moe_dispatch_quantized(x32.data_ptr(), 0, T, 32, k, rows.data_ptr(), 0, codes[1:].data_ptr(),
                                    scales[1:].data_ptr(), s) == 0
    assert (codes[[0, 4, 5, 6, 7]] == 5).all() and (scales[[0, 4, 5, 6, 7]] == 5).all()
    assert (codes[3] == 0).all() and scales[3] == 1 and (codes[1] != 5).any()


def test_rows_past_32_bit_offsets():
    """Rows whose byte and element offsets pass 2^32."""
    T, k, H, E = 40000, 16, 7168, 64
    g = np.random.default_rng(5)
    plan = mxq.moe_plan(i32(random_experts(g, T, k, E, 0.0)), E)
    x = values(g, (T, 64), "bf16").repeat(1, H // 64).contiguous()
    x += torch.arange(H, device=dev(), dtype=torch.float32).to(torch.bfloat16) / 64
    out = mxq.moe_dispatch(x, plan)
    assert out.numel() > 2 ** 32
    at = torch.from_numpy(np.concatenate([[0, T * k - 1], g.integers(0, T * k, 2000)])).to(dev())
    assert torch.equal(out[at], x[plan.slots[at].long() // k])
    w = torch.full((T, k), 1.0 / 16, device=dev())
    back = mxq.moe_combine(out, w, plan)
    assert torch.equal(back, x)                            # 16 equal rows, each times 1/16: exact
    leaf = out.requires_grad_(True)
    gy, = torch.autograd.grad(mxq.moe_combine(leaf, w, plan), leaf, x)
    assert torch.equal(gy[at], x[plan.slots[at].long() // k] / 16)


def test_rows_refusals():
    e = torch.zeros(4, 2, dtype=torch.int32, device=dev())
    plan = mxq.moe_plan(e, 4)
    x, y, w = torch.zeros(4, 32, device=dev()), torch.zeros(8, 32, device=dev()), torch.zeros(4, 2, device=dev())
    for call in (lambda: mxq.moe_dispatch(x[:3], plan), lambda: mxq.moe_combine(y[:7], w, plan),
                 lambda: mxq.moe_combine(y, w[:, :1], plan), lambda: mxq.moe_dispatch(x.view(2, 2, 32), plan),
                 lambda: mxq.moe_dispatch_quantized(x[:, :31], plan, "fp8"),
                 lambda: mxq.moe_dispatch_quantized(x, plan, "nvfp4")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mxq.moe_combine(y, w.half(), plan), lambda: mxq.moe_dispatch(x.double(), plan),
                 lambda: mxq.moe_dispatch(x, mxq.MoEPlan(plan.offs, plan.rows.long(), plan.slots))):
        with pytest.raises(TypeError):
            call()
