"""GPU parity of the router (moe_route) and its gradient against the float64
oracle: choices equal, weights and gradients to the rounding of their type."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from oracle import moe
from tests.gpu_util import DTYPES, dev
from tests.moe_util import U, assert_rounded, f64, i32, values

pytestmark = pytest.mark.gpu


def check(x, k, dtype="f32", bias=None, mask=None, grad=True, **kw):
    """Forward and backward of x [T, E] on the device against the oracle."""
    g = np.random.default_rng(x.shape[0] * 1000 + x.shape[1])
    score, renorm, scale = kw.get("score", "softmax"), kw.get("renormalize", True), kw.get("scale", 1.0)
    leaf = x.detach().clone().requires_grad_(True)
    bt = None if bias is None else torch.from_numpy(bias).to(dev())
    mt = None if mask is None else torch.from_numpy(mask).to(dev())
    w, e = mxq.moe_route(leaf, k, bias=bt, token_mask=mt, **kw)
    want_w, want_e = moe.route(f64(x), k, bias=None if bias is None else bias.astype(np.float64), token_mask=mask, **kw)
    assert w.dtype == torch.float32 and e.dtype == torch.int32 and not e.requires_grad
    assert np.array_equal(e.cpu().numpy(), want_e), "experts"
    # one rounding to fp32; a softmax's sum may hold fp32 exponentials, each off by 2 ulp: 4 roundings more
    assert_rounded(w, want_w, "f32", 4 * U * np.abs(want_w), "weights")
    w2, e2 = mxq.moe_route(x.detach(), k, bias=bt, token_mask=mt, **kw)
    assert torch.equal(w, w2) and torch.equal(e, e2), "the call without a gradient gives the same"
    if grad:
        gw = g.standard_normal(want_w.shape).astype(np.float32)
        got, = torch.autograd.grad(w, leaf, torch.from_numpy(gw).to(dev()))
        assert got.dtype == x.dtype
        xs = f64(x)
        want = moe.route_grad(xs, want_e, gw.astype(np.float64), score, renorm, scale)
        # the same 4 roundings on each score, and on the sum that a softmax takes off (at most scale * max |g| / S * S)
        top = np.zeros(xs.shape)
        for t in range(xs.shape[0]):
            s = np.nan_to_num(moe.scores(xs[t], score), nan=0.0)
            live = [i for i in want_e[t] if i >= 0]
            total = s[live].sum() if renorm and live else 1.0
            top[t] = 3 * abs(scale) * np.abs(gw[t]).max() / max(total, 1e-300) * s if live else 0.0
        assert_rounded(got, want, dtype, 8 * U * top, "grad_logits")


SIZES = [(1, 8, 2), (3, 60, 4), (5, 64, 8), (64, 256, 8), (65, 256, 1), (7, 384, 6), (4, 1024, 32), (2, 33, 32),
         (9, 1, 1), (6, 17, 17), (1, 512, 9), (130, 128, 8), (5, 1000, 3), (7, 100, 20),
         (5, 300, 8), (6, 512, 16), (3, 500, 24)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_sizes(T, E, k, score):
    g = np.random.default_rng(T + E + k)
    x = values(g, (T, E), "f32", 1.5)
    check(x, k, score=score, renormalize=True, scale=2.5)
    check(x, k, score=score, renormalize=False)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    check(x, k, score=score, bias=bias, renormalize=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_types_with_many_ties(dtype, score):
    """16-bit logits repeat within a token; equal ones go to the lower expert, with or without a constant bias."""
    g = np.random.default_rng(11)
    x = values(g, (96, 256), dtype)
    x[3] = 0.0
    x[4] = -0.0
    x[5, ::2] = -0.0
    check(x, 8, dtype, score=score)
    check(x, 8, dtype, score=score, bias=np.zeros(256, np.float32))
    check(x, 8, dtype, score=score, bias=np.full(256, 0.25, np.float32), groups=8, top_groups=3)
    check(x, 8, dtype, score=score, groups=8, top_groups=3, renormalize=False)


def test_route_near_ties_are_decided_in_fp64():
    """Keys that differ by less than fp32 holds: logits one ulp apart under equal biases, and biases that lift
    different scores to within 1e-9 of each other."""
    g = np.random.default_rng(12)
    x = np.full((64, 256), 2.0, np.float32)
    steps = g.integers(0, 3, (64, 256))
    x = (x.view(np.int32) + steps.astype(np.int32)).view(np.float32)
    check(torch.from_numpy(x).to(dev()), 8, score="sigmoid", bias=np.full(256, 0.5, np.float32))
    logits = g.standard_normal((64, 256)).astype(np.float32)
    s = moe.sigmoid(logits[0].astype(np.float64))
    bias = (1.5 - s).astype(np.float32)                  # token 0's keys are all 1.5 but for fp32's rounding of the bias
    check(torch.from_numpy(logits).to(dev()), 8, score="sigmoid", bias=bias)
    check(torch.from_numpy(logits).to(dev()), 8, score="sigmoid", bias=bias, groups=8, top_groups=4)


GROUPS = [(64, 4, 2, 8, 2), (256, 8, 4, 8, 2), (160, 8, 3, 6, 1), (256, 8, 1, 8, 2), (60, 12, 5, 4, 2), (64, 64, 8, 8, 2),
          (1024, 64, 4, 8, 2), (21, 3, 2, 5, 2), (256, 4, 4, 8, 2), (12, 6, 1, 4, 2), (512, 16, 3, 8, 1), (512, 4, 2, 8, 2), (384, 8, 4, 8, 2), (320, 5, 2, 6, 2),
          (130, 13, 4, 8, 2), (1000, 8, 3, 8, 2), (130, 13, 2, 32, 1), (480, 3, 2, 8, 2), (240, 5, 2, 8, 2), (96, 8, 3, 8, 2),
          (60, 4, 2, 16, 2), (405, 9, 4, 8, 2), (510, 3, 1, 8, 1), (15, 15, 4, 4, 2), (42, 14, 5, 9, 1), (155, 5, 2, 8, 2)]


@pytest.mark.parametrize("E,groups,top_groups,k,best", GROUPS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(E, groups, top_groups, k, best, score):
    """More places than the kept groups hold leave -1 behind."""
    g = np.random.default_rng(E + groups)
    x = values(g, (70, E), "f32", 1.5)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    check(x, k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_best=best)
    check(x, k, score=score, groups=groups, top_groups=top_groups, group_best=best, renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_and_empty(score):
    """Masked tokens hold NaN; experts are closed by logits or biases of -inf; a row with no expert left."""
    g = np.random.default_rng(13)
    x = values(g, (40, 64), "f32")
    mask = g.random(40) > 0.3
    mask[:2] = [False, True]
    x[torch.from_numpy(~mask).to(dev())] = float("nan")
    x[1] = float("-inf")
    x[2, 5:] = float("-inf")
    x[:, 7] = float("-inf")
    x[3, 9] = float("nan")
    x[4, ::2] = torch.finfo(torch.float32).min
    x[5, 2:] = torch.finfo(torch.float32).min
    bias = (0.1 * g.standard_normal(64)).astype(np.float32)
    bias[20:30] = -np.inf
    for kw in (dict(), dict(bias=bias), dict(bias=bias, groups=8, top_groups=2), dict(groups=8, top_groups=8)):
        check(x, 8, score=score, mask=mask, **kw)
        check(x, 8, score=score, mask=mask, renormalize=False, **kw)
    none = np.zeros(40, bool)
    check(x, 8, score=score, mask=none)


@pytest.mark.parametrize("E,k,kw", [(5, 2, dict()), (60, 5, dict()), (128, 6, dict(groups=8, top_groups=3)), (256, 8, dict()),
                                    (256, 7, dict(groups=8, top_groups=4)), (384, 5, dict()), (512, 8, dict()),
                                    (700, 9, dict()), (130, 6, dict(groups=13, top_groups=5)), (96, 20, dict())])
@pytest.mark.parametrize("share", [0.1, 0.6])
def test_route_nan_logits_and_biases(E, k, kw, share):
    """NaN in any place of the logits or the bias closes that expert and disturbs no other."""
    g = np.random.default_rng(E + k)
    x = values(g, (70, E), "f32")
    x[torch.from_numpy(g.random((70, E)) < share).to(dev())] = float("nan")
    bias = (0.1 * g.standard_normal(E)).astype(np.float32)
    bias[g.random(E) < 0.2] = np.nan
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            want_w, want_e = moe.route(f64(x), k, score, bias=None if b is None else b.astype(np.float64), **kw)
            w, e = mxq.moe_route(x, k, score=score, bias=None if b is None else torch.from_numpy(b).to(dev()), **kw)
            assert np.array_equal(e.cpu().numpy(), want_e)
            assert_rounded(w, want_w, "f32", 4 * U * want_w, "weights")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_far_values(score):
    """Logits far from 0: scores that round to 1 or vanish in fp32 keep their order and their weights."""
    x = torch.tensor([[90.0, 95.0, -200.0, 30.0, 0.0, -90.0, -91.0, 95.0],
                      [-300.0, -301.0, -302.0, -303.0, -304.0, -305.0, -306.0, -307.0]], device=dev())
    check(x, 3, score=score, grad=False)
    check(x, 8, score=score, renormalize=False, grad=False)
    bias = np.array([0, 0, 3, 0, 0, 3, 3, 0], np.float32)        # the choice falls on logits far below the largest
    check(x, 3, score=score, bias=bias)
    wide = torch.cat([x, x - 1, x - 2], 1)
    check(wide, 20, score=score, bias=np.concatenate([bias] * 3))
    low = torch.full((3, 130), torch.finfo(torch.float16).min, device=dev()).half()
    low[:, 7] = 0.0
    check(low, 5, "f16", score=score, bias=(np.arange(130) == 90).astype(np.float32) * 9, groups=13, top_groups=2)


def test_route_gradient_of_a_peaked_softmax():
    """One score near 1: the gradient s (1 - s) of its logit keeps the accuracy of the others' sum.  Exponentials off by
    4 u, their sum by as much, the products' and the result's roundings: 16 u, relative.  Absolute: z, s and u s are fp64
    values next to 1, here and in the oracle alike: each of the E - 1 additions in z, the quotient, the product and the
    difference round by up to 2^-53, on both sides."""
    x = torch.zeros(30, 60, device=dev())
    x[:, 11] = torch.linspace(2, 30, 30, device=dev())
    x.requires_grad_(True)
    for E in (60, 300):
        leaf = torch.nn.functional.pad(x.detach(), (0, E - 60)).requires_grad_(True)
        w, e = mxq.moe_route(leaf, 1, renormalize=False)
        assert (e == 11).all()
        g, = torch.autograd.grad(w.sum(), leaf)
        want = moe.route_grad(f64(leaf), e.cpu().numpy(), np.ones((30, 1)), "softmax", False, 1.0)
        off = np.abs(f64(g) - want)
        assert (off <= 16 * U * np.abs(want) + 2 * (E + 2) * 2.0 ** -53).all(), (off / np.abs(want)).max()


def many(g, T, E, dtype="f32", distinct=40):
    """T tokens' logits with `distinct` different rows in a random order, so that the oracle stays quick."""
    x = values(g, (distinct, E), dtype, 1.5)
    return x, torch.from_numpy(g.integers(0, distinct, T)).to(dev())


MANY = [(4096, 256, 8, dict(groups=8, top_groups=4)), (5001, 256, 8, dict()), (2050, 60, 4, dict()), (3000, 64, 16, dict()),
        (2048, 128, 1, dict(groups=4, top_groups=1)), (2049, 17, 3, dict()), (2500, 96, 6, dict(groups=12, top_groups=5)),
        (2500, 240, 8, dict(groups=5, top_groups=2)), (2300, 256, 16, dict(groups=2, top_groups=1, group_best=1)),
        (2100, 384, 8, dict(groups=8, top_groups=3)), (2100, 200, 17, dict()), (2100, 130, 8, dict(groups=13, top_groups=4)),
        (2100, 512, 8, dict(groups=16, top_groups=5)), (2100, 500, 10, dict()),
        (2200, 160, 6, dict(groups=8, top_groups=3, group_best=1)), (2100, 60, 4, dict(groups=4, top_groups=2))]


@pytest.mark.parametrize("T,E,k,kw", MANY)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_many_tokens(T, E, k, kw, score, dtype):
    """The choice of a token does not hang on how many there are, nor on its neighbours: every row of a large call
    equals the oracle's answer for it, with ties, closed experts, masked and NaN rows among them."""
    g = np.random.default_rng(T + E)
    x, order = many(g, T, E, dtype)
    x[3] = 0.5
    x[4, 1:] = float("-inf")
    x[5, ::3] = float("-inf")
    x[6] = float("-inf")
    x[7, 5] = float("nan")
    x[8] = torch.round(x[8])
    x[9, ::2] = torch.finfo(x.dtype).min                 # masked with the type's lowest value: still finite logits
    x[10, : E - min(k, E) + 1] = torch.finfo(x.dtype).min
    x[11, 1:] = -1e9
    for bias in (None, (0.1 * g.standard_normal(E)).astype(np.float32), np.zeros(E, np.float32)):
        args = dict(score=score, renormalize=bias is not None, **kw)
        want_w, want_e = moe.route(f64(x), k, bias=None if bias is None else bias.astype(np.float64), **args)
        mask = torch.from_numpy(g.random(T) > 0.1).to(dev())
        w, e = mxq.moe_route(x[order], k, bias=None if bias is None else torch.from_numpy(bias).to(dev()),
                             token_mask=mask, **args)
        on, at = mask.cpu().numpy(), order.cpu().numpy()
        assert np.array_equal(e.cpu().numpy(), np.where(on[:, None], want_e[at], -1))
        want = np.where(on[:, None], want_w[at], 0.0)
        assert_rounded(w, want, "f32", 4 * U * np.abs(want), "weights")


@pytest.mark.parametrize("E,k,kw", [(256, 8, {}), (1000, 24, {}), (300, 6, {"groups": 60, "top_groups": 3})])
def test_route_past_32_bit_offsets(E, k, kw):
    """Tokens whose logits lie past 2^31 elements and 2^32 bytes: what the same tokens give alone."""
    T = 2 ** 31 // E + 70_000
    x = torch.randn(T, E, device=dev(), dtype=torch.bfloat16, generator=torch.Generator(dev()).manual_seed(9))
    at = torch.tensor([0, T // 2, T - 70_000, T - 69_999, T - 2, T - 1], device=dev())
    leaf, few = x.requires_grad_(True), x.detach()[at].requires_grad_(True)
    w, e = mxq.moe_route(leaf, k, **kw)
    want_w, want_e = mxq.moe_route(few, k, **kw)
    assert torch.equal(w[at], want_w) and torch.equal(e[at], want_e)
    gw = torch.randn(T, k, device=dev())
    got, = torch.autograd.grad(w, leaf, gw)
    want, = torch.autograd.grad(want_w, few, gw[at])
    assert torch.equal(got[at], want)


def test_route_strided_and_misaligned_logits():
    g = np.random.default_rng(14)
    base = values(g, (33, 2 * 60 + 1), "bf16")
    check(base[:, 1:61], 4, "bf16")
    check(base[:, 1::2], 4, "bf16", score="sigmoid")
    flat = values(g, (33 * 60 + 1,), "bf16")[1:].view(33, 60)      # contiguous, 2-byte aligned
    check(flat, 4, "bf16")
    assert mxq.moe_route(base[:0, :60], 4)[1].shape == (0, 4)


def test_route_gradient_with_out_of_range_index():
    """Index values outside the experts count as places without one (entry point called directly)."""
    from nvfp4_quantization_grouped_amd import _lib
    g = np.random.default_rng(15)
    x = values(g, (5, 16), "f32")
    idx = np.array([[0, 16, 3], [-1, -7, 2 ** 31 - 1], [15, -1, 1], [-2 ** 31, 4, 5], [2, 1, 0]], np.int32)
    gw = g.standard_normal((5, 3)).astype(np.float32)
    it, gt, out = i32(idx), torch.from_numpy(gw).to(dev()), torch.full_like(x, 7.0)
    st = _lib.moe_lib().moe_route_bwd(x.data_ptr(), 0, 5, 16, 3, 1, 1, 1.0, it.data_ptr(), gt.data_ptr(),
                                      out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want = moe.route_grad(f64(x), idx, gw.astype(np.float64), "sigmoid", True, 1.0)
    assert_rounded(out, want, "f32", 8 * U * np.abs(gw).max() * 8, "grad")


def test_route_near_ties_among_many_tokens():
    """The near ties above where four tokens share a wave, in every third token, the others far from ties."""
    g = np.random.default_rng(21)
    distinct = 12
    x = (1.5 * g.standard_normal((distinct, 256))).astype(np.float32)
    for r in range(0, distinct, 3):                      # within two ulps of each other
        x[r] = (np.full(256, 2.0, np.float32).view(np.int32) + g.integers(0, 3, 256).astype(np.int32)).view(np.float32)
    x[1] = g.standard_normal(256)
    bias = (1.5 - moe.sigmoid(x[1].astype(np.float64))).astype(np.float32)
    order = g.integers(0, distinct, 2304)
    at = torch.from_numpy(x[order]).to(dev())
    for b in (bias, np.full(256, 0.5, np.float32)):
        for kw in (dict(), dict(groups=8, top_groups=4), dict(groups=8, top_groups=4, group_best=1)):
            for score in ("sigmoid", "softmax"):
                w, e = mxq.moe_route(at, 8, score=score, bias=torch.from_numpy(b).to(dev()), **kw)
                want_w, want_e = moe.route(x.astype(np.float64), 8, score, bias=b.astype(np.float64), **kw)
                assert np.array_equal(e.cpu().numpy(), want_e[order])
                assert_rounded(w, want_w[order], "f32", 4 * U * want_w[order], "weights")


@pytest.mark.parametrize("T", [3, 2050])
def test_route_infinite_logits(T):
    """A logit of +inf is a sigmoid score of 1 and comes before every finite logit."""
    g = np.random.default_rng(22)
    x = g.standard_normal((5, 64)).astype(np.float32)
    x[0, 7], x[1, [3, 60]] = np.inf, np.inf
    x[2] = np.inf
    order = np.arange(T) % 5
    at = torch.from_numpy(x[order]).to(dev())
    for kw in (dict(), dict(bias=(0.1 * g.standard_normal(64)).astype(np.float32))):
        want_w, want_e = moe.route(x.astype(np.float64), 6, "sigmoid", **kw)
        w, e = mxq.moe_route(at, 6, score="sigmoid", **{k: torch.from_numpy(v).to(dev()) for k, v in kw.items()})
        assert np.array_equal(e.cpu().numpy(), want_e[order])
        assert_rounded(w, want_w[order], "f32", 4 * U * want_w[order], "weights")


def test_route_second_derivatives_are_refused():
    x = torch.randn(4, 16, device=dev(), requires_grad=True)
    w, _ = mxq.moe_route(x, 4)
    g, = torch.autograd.grad(w.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
    w, e = mxq.moe_route(x, 4)
    assert torch.autograd.grad(w.sum() * 0 + x.sum(), x)[0].shape == x.shape


def test_route_refusals():
    x = torch.zeros(4, 64, device=dev())
    for bad in (dict(top_k=0), dict(top_k=33), dict(top_k=65)):
        with pytest.raises(ValueError):
            mxq.moe_route(x, **bad)
    with pytest.raises(mxq.MxqError):
        mxq.moe_route(x, 4, groups=7)
    with pytest.raises(mxq.MxqError):
        mxq.moe_route(torch.zeros(4, 1025, device=dev()), 4)
    with pytest.raises(TypeError):
        mxq.moe_route(x, 4, bias=torch.zeros(64, device=dev(), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        mxq.moe_route(x, 4, token_mask=torch.zeros(5, device=dev(), dtype=torch.bool))
    with pytest.raises(TypeError):
        mxq.moe_route(x.double(), 4)
    with pytest.raises(ValueError):
        mxq.moe_route(x.view(2, 2, 64), 4)


def test_route_in_a_graph_and_on_another_stream():
    g = np.random.default_rng(16)
    x = values(g, (257, 256), "f32")
    bias = torch.from_numpy((0.1 * g.standard_normal(256)).astype(np.float32)).to(dev())
    kw = dict(score="sigmoid", bias=bias, groups=8, top_groups=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    gw = values(g, (257, 8), "f32")
    static = x.clone()
    with torch.cuda.stream(side):
        mxq.moe_route(static, 8, **kw)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        leaf = static.detach().requires_grad_(True)
        w, e = mxq.moe_route(leaf, 8, **kw)
        grad, = torch.autograd.grad(w, leaf, gw)
    for seed in range(4):
        new = values(np.random.default_rng(seed), (257, 256), "f32")
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        leaf2 = new.clone().requires_grad_(True)
        w2, e2 = mxq.moe_route(leaf2, 8, **kw)
        g2, = torch.autograd.grad(w2, leaf2, gw)
        assert torch.equal(w, w2) and torch.equal(e, e2) and torch.equal(grad, g2)
