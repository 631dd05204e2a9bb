"""GPU parity of the router under biases far from the scores: experts pinned
with +inf, and closed with the lowest values of fp32, in each of the three
kernels (16 lanes a token, a wave a token, fp64 keys throughout), against the
float64 oracle."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from oracle import moe
from tests.gpu_util import dev
from tests.moe_util import U, assert_rounded, f64, values
from tests.test_gpu_moe_route import check

pytestmark = pytest.mark.gpu

# experts, places, groups: 16 lanes a token (one group; whole and dealt-out groups), a wave a token (more than 16 places,
# more than 512 experts, more than 16 groups), fp64 keys throughout (groups of 5 experts, 8 a lane)
SHAPES = [(256, 8, dict()), (60, 4, dict()), (17, 16, dict()), (256, 8, dict(groups=8, top_groups=4)),
          (160, 6, dict(groups=8, top_groups=3)), (60, 4, dict(groups=4, top_groups=2, group_best=1)),
          (256, 20, dict()), (60, 20, dict()), (700, 9, dict()), (256, 20, dict(groups=8, top_groups=4)),
          (1024, 8, dict(groups=2, top_groups=1)), (64, 20, dict(groups=32, top_groups=20)),
          (320, 8, dict(groups=64, top_groups=5))]


def pinned(E, k, groups):
    """Sets of experts for a bias of +inf: fewer than the places, as many, more, a whole group, all of them."""
    g = np.random.default_rng(E + k)
    size = E // groups
    sets = [g.permutation(E)[:n] for n in (1, 2, k - 1, k, k + 1, 3 * k) if 0 < n <= E]
    return sets + [np.arange(E - size, E), np.array([0, E - 1]), np.arange(E)]


@pytest.mark.parametrize("E,k,kw", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_biases_of_plus_infinity(E, k, kw, score):
    """Pinned experts come first, in index order, and pin their groups; the rest follow as without them."""
    g = np.random.default_rng(E)
    x = values(g, (9, E), "f32", 1.5)
    x[1] = 0.25
    x[2, ::3] = float("-inf")
    x[3, 1::2] = float("nan")
    for i, which in enumerate(pinned(E, k, kw.get("groups", 1))):
        bias = (0.1 * g.standard_normal(E)).astype(np.float32) if i % 2 else np.zeros(E, np.float32)
        bias[which] = np.inf
        check(x, k, score=score, bias=bias, renormalize=i % 3 > 0, grad=False, **kw)
        bias[g.permutation(E)[: E // 4]] = -np.inf
        check(x, k, score=score, bias=bias, grad=False, **kw)


def check_between_guards(x, k, bias, score, **kw):
    """The router on x [T, E] and bias [E] that lie between logits of 1e30 and biases of +inf: an expert read past either
    end, or taken from another token's, would be chosen."""
    T, E = x.shape
    logits = torch.full((T + 2, E), 1e30, device=dev())
    logits[1:T + 1] = x
    biases = torch.full((3 * E,), float("inf"), device=dev())
    biases[E:2 * E] = torch.from_numpy(bias).to(dev())
    w, e = mxq.moe_route(logits[1:T + 1], k, score=score, bias=biases[E:2 * E], **kw)
    want_w, want_e = moe.route(f64(x), k, score, bias=bias.astype(np.float64), **kw)
    assert np.array_equal(e.cpu().numpy(), want_e)
    assert_rounded(w, want_w, "f32", 4 * U * np.abs(want_w), "weights")


CLOSED = SHAPES + [(96, 5, dict(groups=8, top_groups=3)), (130, 8, dict(groups=13, top_groups=4)),
                   (64, 20, dict()), (33, 20, dict())]


@pytest.mark.parametrize("E,k,kw", CLOSED)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("low", [float(np.finfo(np.float32).min), -3e38])
def test_route_biases_of_the_lowest_values(E, k, kw, score, low):
    """Experts closed with the lowest values are taken when no other is left, and no place that holds no expert ever is:
    every other expert, all but few, and groups of which all experts or all but one are closed."""
    g = np.random.default_rng(E + k)
    x = values(g, (11, E), "f32", 1.5)
    x[1] = 0.25
    x[2, ::3] = float("-inf")
    groups, top = kw.get("groups", 1), kw.get("top_groups", 1)
    size = E // groups
    base = (0.1 * g.standard_normal(E)).astype(np.float32)
    shut = [np.arange(0, E, 2), g.permutation(E)[k // 2:]] if groups == 1 else []
    for n in range(1, groups - top + 1, max(1, (groups - top) // 3)):          # top groups at least stay open
        at = g.permutation(groups)[:n]
        if groups - 1 not in at:
            at[0] = groups - 1                                                 # the last one, at the end of the row
        whole = np.concatenate([np.arange(q * size, (q + 1) * size) for q in at])
        shut += [whole, np.array([e for e in whole if e % size != size // 2])]
    for which in shut:
        bias = base.copy()
        bias[which] = low
        check_between_guards(x, k, bias, score, **kw)
        check_between_guards(x, k, bias, score, renormalize=False, **kw)


GROUPED = [(256, 8, 8), (160, 6, 8), (60, 4, 4), (256, 20, 8), (1024, 9, 4), (320, 8, 64)]      # experts, places, groups


@pytest.mark.parametrize("E,k,groups", GROUPED)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("sign", [1, -1])
def test_route_group_values_past_the_range_of_fp32(E, k, groups, score, sign):
    """Two keys whose sum no fp32 value holds still give their group its place: each group with a bias of its own near
    either end of the range, some equal, one group without any expert."""
    g = np.random.default_rng(E + groups)
    x = values(g, (8, E), "f32", 1.5)
    size = E // groups
    x[:, :size] = float("-inf")
    for top in (1, 2, groups // 2, groups - 1, groups):
        for steps in (g.permutation(groups), g.integers(0, 3, groups)):
            bias = np.repeat(sign * (1.8e38 + 1.6e38 * steps / groups), size).astype(np.float32)
            check_between_guards(x, k, bias, score, groups=groups, top_groups=top)
            bias[-size:] = 0.5                             # one group of ordinary biases
            check_between_guards(x, k, bias, score, groups=groups, top_groups=top)
