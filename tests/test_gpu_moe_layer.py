"""The operators of the routed-expert layer run together, as a layer uses them
(mxfp4_moe and its parts), against the float64 oracle: outputs, gradients,
captured graphs and other streams."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
import oracle
import synth
from oracle import moe
from tests.gpu_util import dev
from tests.moe_util import f64, values
from tests.test_gpu_grouped_mm import gpu_weights

pytestmark = pytest.mark.gpu

E, H, I, K = 8, 512, 512, 4


def layer(seed=0):
    st = synth.streams(seed, 4)
    gu = synth.packed_weights(st[0], st[1], E, 2 * I, H)
    dn = synth.packed_weights(st[2], st[3], E, H, I)
    # both dequantized to unit-sized products: scale bytes lowered by 2^-3
    gu = (gu[0], (gu[1] - 2).astype(np.uint8))
    dn = (dn[0], (dn[1] - 2).astype(np.uint8))
    return gu, dn


def on_gpu(w):
    return gpu_weights(*w)


def bf16(a):
    return oracle.from_dtype_bits(oracle.to_dtype_bits(a, "bf16"), "bf16")


def rel(got, want):
    return np.linalg.norm(f64(got) - want) / np.linalg.norm(want)


def oracle_pass(x, w, e, gu, dn, first, local, go):
    """Forward and gradients with the layer's own roundings to bf16 between its operators."""
    offs, rows, _ = moe.plan(e, first, local)
    xg = moe.dispatch(x, rows)
    a = bf16(oracle.grouped_mm_fwd(xg, gu[0], gu[1], offs))
    h = bf16(moe.swiglu(a))
    h[offs[-1]:] = 0
    y = bf16(oracle.grouped_mm_fwd(h, dn[0], dn[1], offs))
    out = moe.combine(y, w, rows)
    gy, gw = moe.combine_grad(go, y, w, rows)
    gh = bf16(oracle.grouped_mm_bwd_x(bf16(gy), dn[0], dn[1], offs))
    ga = moe.swiglu_grad(moe.kept(a), gh)
    ga[offs[-1]:] = 0
    gx = moe.dispatch_grad(bf16(oracle.grouped_mm_bwd_x(bf16(ga), gu[0], gu[1], offs)), rows)
    return out, gx, gw


# Each operator rounds to bf16 once (relative Frobenius error about 2^-9 / sqrt(3) of its output, at most 2^-8) and the
# products hold 5e-3 by their own tests; the oracle rounds at the same places, so what is left is values that fall to
# the other side of a rounding: 5e-3 a product, 2 products forward, 2 more backward, one 2^-8 a rounding between.
OUT, GRAD = 2 * 5e-3 + 3 * 2.0 ** -8, 4 * 5e-3 + 6 * 2.0 ** -8


@pytest.mark.parametrize("T,first,local", [(1, 0, 8), (75, 0, 8), (300, 2, 4)])
def test_layer_forward_and_gradients(T, first, local):
    g = np.random.default_rng(T)
    gu, dn = layer()
    sl = slice(first, first + local)
    gu, dn = (gu[0][sl], gu[1][sl]), (dn[0][sl], dn[1][sl])
    x = values(g, (T, H), "bf16").requires_grad_(True)
    logits = values(g, (T, E), "f32").requires_grad_(True)
    mask = torch.from_numpy(np.arange(T) % 7 != 3).to(dev())
    weights, experts = mxq.moe_route(logits, K, score="sigmoid", groups=4, top_groups=3, token_mask=mask)
    (gp, gs), (dp, ds) = on_gpu(gu), on_gpu(dn)
    out = mxq.mxfp4_moe(x, weights, experts, gp, gs, dp, ds, num_experts=E, first_expert=first)
    go = values(g, (T, H), "bf16")
    gx, gw, gl = torch.autograd.grad(out, (x, weights, logits), go)
    want, want_x, want_w = oracle_pass(f64(x), f64(weights), experts.cpu().numpy(), gu, dn, first, local, f64(go))
    assert out.shape == (T, H) and out.dtype == torch.bfloat16
    assert rel(out, want) <= OUT and rel(gx, want_x) <= GRAD and rel(gw, want_w) <= GRAD
    want_l = moe.route_grad(f64(logits), experts.cpu().numpy(), f64(gw), "sigmoid")
    assert rel(gl, want_l) <= 1e-6
    if T > 3:
        assert (out[3] == 0).all() and (gl[3] == 0).all() and (gx[3] == 0).all()


@pytest.mark.parametrize("activations", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T", [0, 5])
def test_layer_with_no_row_to_serve(T, activations):
    """No token, or tokens that go nowhere: zeros, and zero gradients."""
    (gp, gs), (dp, ds) = (on_gpu(w) for w in layer())
    x = torch.ones(T, H, dtype=torch.bfloat16, device=dev(), requires_grad=activations == "bf16")
    w = torch.full((T, K), float("nan"), device=dev(), requires_grad=activations == "bf16")
    e = torch.full((T, K), -1, dtype=torch.int32, device=dev())
    out = mxq.mxfp4_moe(x, w, e, gp, gs, dp, ds, activations=activations)
    assert out.shape == (T, H) and not out.any()
    if activations == "bf16":
        gx, gw = torch.autograd.grad(out, (x, w), torch.ones_like(out))
        assert gx.shape == x.shape and gw.shape == w.shape and not gx.any() and not gw.any()


@pytest.mark.parametrize("activations", ["fp8", "mxfp4"])
def test_layer_with_low_bit_activations(activations):
    """Equal, bit for bit, to the layer put together from dispatch and the products that quantize themselves."""
    g = np.random.default_rng(3)
    (gp, gs), (dp, ds) = (on_gpu(w) for w in layer())
    x = values(g, (90, H), "bf16")
    w, e = mxq.moe_route(values(g, (90, E), "f32"), K)
    out = mxq.mxfp4_moe(x, w, e, gp, gs, dp, ds, activations=activations)
    mm = mxq.mxfp4_grouped_mm_fwd_w4a8 if activations == "fp8" else mxq.mxfp4_grouped_mm_fwd_w4a4
    plan = mxq.moe_plan(e, E)
    h = mxq.swiglu(mm(mxq.moe_dispatch(x, plan), gp, gs, plan.offs), plan.offs)
    assert torch.equal(out, mxq.moe_combine(mm(h, dp, ds, plan.offs), w, plan))
    with pytest.raises(ValueError):
        mxq.mxfp4_moe(x.requires_grad_(True), w, e, gp, gs, dp, ds, activations=activations)


def test_layer_in_a_graph():
    """Forward and backward captured and replayed between eager passes, every replay against the eager result."""
    g = np.random.default_rng(4)
    (gp, gs), (dp, ds) = (on_gpu(w) for w in layer())
    T = 64
    x, logits, go = values(g, (T, H), "bf16"), values(g, (T, E), "f32"), values(g, (T, H), "bf16")

    def step(x, logits):
        x, logits = x.detach().requires_grad_(True), logits.detach().requires_grad_(True)
        w, e = mxq.moe_route(logits, K)
        out = mxq.mxfp4_moe(x, w, e, gp, gs, dp, ds)
        return (out, *torch.autograd.grad(out, (x, logits), go))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, logits)
    side.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        first = step(x, logits)
    with torch.cuda.graph(other, stream=side):             # a second graph of the same calls, replayed in turn
        second = step(x, logits)
    for seed in range(4):
        r = np.random.default_rng(100 + seed)
        x.copy_(values(r, (T, H), "bf16"))
        logits.copy_(values(r, (T, E), "f32"))
        graph.replay()
        want = step(x, logits)
        other.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(first, second, want):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_rows_in_a_graph():
    """The two-launch order of many slots, the streams and their gradients captured; replays between eager passes over
    other assignments, every replay against the eager result."""
    g = np.random.default_rng(8)
    T, k, n, F = 5000, 5, 40, 192
    e = torch.from_numpy(g.integers(-1, n, (T, k)).astype(np.int32)).to(dev())
    x, w, go = values(g, (T, F), "bf16"), values(g, (T, k), "f32"), values(g, (T, F // 2), "bf16")

    def step(e, x, w):
        x, w = x.detach().requires_grad_(True), w.detach().requires_grad_(True)
        plan = mxq.moe_plan(e, n)
        codes, scales = mxq.moe_dispatch_quantized(x, plan, "fp8")
        out = mxq.moe_combine(mxq.swiglu(mxq.moe_dispatch(x, plan), plan.offs), w, plan)
        return (*plan, codes, scales, out, *torch.autograd.grad(out, (x, w), go))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(e, x, w)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step(e, x, w)
    for seed in range(4):
        r = np.random.default_rng(200 + seed)
        e.copy_(torch.from_numpy(r.integers(-1, n, (T, k)).astype(np.int32)))
        x.copy_(values(r, (T, F), "bf16"))
        w.copy_(values(r, (T, k), "f32"))
        graph.replay()
        want = step(e, x, w)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_layer_on_two_streams_at_once():
    """Two plans and their rows at the same time, each on its own stream with its own workspace."""
    g = np.random.default_rng(5)
    T, k, n = 20000, 4, 64
    es = [torch.from_numpy(g.integers(-1, n, (T, k)).astype(np.int32)).to(dev()) for _ in range(2)]
    xs = [values(g, (T, 64), "bf16") for _ in range(2)]
    want = [mxq.moe_dispatch(x, mxq.moe_plan(e, n)) for x, e in zip(xs, es)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, x, e in zip(streams, xs, es):
            with torch.cuda.stream(s):
                got.append(mxq.moe_dispatch(x, mxq.moe_plan(e, n)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layer_gradcheck_by_differences():
    """The composed fp32 parts (router, dispatch, swiglu with the input kept whole, combine) against central
    differences of their own forward, along random directions."""
    g = np.random.default_rng(6)
    T, F = 12, 64
    x, logits = values(g, (T, F), "f32"), values(g, (T, 6), "f32")
    w0, e0 = mxq.moe_route(logits, 2)
    plan = mxq.moe_plan(e0, 6)
    go = values(g, (T, F // 2), "f32")

    def f(x, logits):
        w, e = mxq.moe_route(logits, 2)
        return mxq.moe_combine(mxq.swiglu(mxq.moe_dispatch(x, plan), plan.offs, checkpoint=None), w, plan), e

    xl, ll = x.clone().requires_grad_(True), logits.clone().requires_grad_(True)
    gx, gl = torch.autograd.grad(f(xl, ll)[0], (xl, ll), go)
    h = 2.0 ** -9
    for k in range(4):
        dx, dl = values(g, (T, F), "f32"), values(g, (T, 6), "f32") * 0.25
        hi, eh = f(x + h * dx, logits + h * dl)
        lo, el = f(x - h * dx, logits - h * dl)
        assert torch.equal(eh, e0) and torch.equal(el, e0)
        diff = float(((hi.double() - lo.double()) * go.double()).sum() / (2 * h))
        want = float((gx.double() * dx.double()).sum() + (gl.double() * dl.double()).sum())
        # fp32 values of size 1, some 2^8.6 of them, each off by at most 8 roundings, over 2 h: 2^-24+3+8.6+8 = 2^-4.4
        # at worst and 2^-9 as independent errors; third derivatives of size 1 times h^2 / 6: 2^-12 of the sum of
        # 2^8.6 terms of size 1, 2^-3.4 at worst
        assert abs(diff - want) < 2.0 ** -4.4 + 2.0 ** -3.4
