"""The router with a wave a token where that form's own steps decide: groups over
one lane, several and 32 of them, lane counts that are no power of two, and keys
that fp32 does not tell apart.  Sizes that the 16-lane form does not take: more
than 16 places, more than 512 experts, or more than 16 groups."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from oracle import moe
from tests.gpu_util import dev
from tests.moe_util import U, assert_rounded, f64, values
from tests.test_gpu_moe_route import check

pytestmark = pytest.mark.gpu

# experts, places, groups, top_groups                 lanes a group x experts a lane
WIDE = [(256, 20, 8, 4),                            # 8 x 4
        (1024, 8, 8, 3),                            # 8 x 16
        (1024, 32, 2, 1),                           # 32 x 16
        (960, 10, 3, 2),                            # 20 x 16
        (960, 17, 5, 2),                            # 12 x 16
        (64, 24, 4, 2),                             # 16 x 1
        (48, 18, 16, 9),                            # 3 x 1
        (64, 5, 32, 7),                             # 2 x 1
        (768, 12, 48, 20),                          # 1 x 16
        (600, 20, 3, 1),                            # groups of 200 at 16 a lane: fp64 keys throughout
        (700, 9, 1, 1), (256, 24, 1, 1), (1024, 32, 1, 1), (40, 32, 1, 1)]


@pytest.mark.parametrize("E,k,groups,top", WIDE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
def test_wide_route(E, k, groups, top, score, best):
    g = np.random.default_rng(E + k)
    x = values(g, (21, E), "f32", 1.5)
    x[1] = 0.5
    x[2, ::3] = float("-inf")
    x[3, 1:] = float("-inf")
    x[4, ::2] = float("nan")
    x[5] = torch.round(x[5])
    x[6, ::2] = torch.finfo(torch.float32).min
    kw = dict(score=score, groups=groups, top_groups=top, group_best=best)
    check(x, k, bias=(0.1 * g.standard_normal(E)).astype(np.float32), grad=False, **kw)
    check(x, k, renormalize=False, grad=False, **kw)
    check(x.bfloat16(), k, "bf16", bias=np.zeros(E, np.float32), grad=False, **kw)


@pytest.mark.parametrize("E,k,groups,top", WIDE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
def test_wide_route_near_ties(E, k, groups, top, score, best):
    """Logits within two ulps of each other under equal biases; biases that lift different scores to within an fp32
    rounding of each other; groups that are copies of each other but for one ulp of one logit."""
    g = np.random.default_rng(E + 7 * k)
    ulps = (np.full((12, E), 2.0, np.float32).view(np.int32) + g.integers(0, 3, (12, E)).astype(np.int32)).view(np.float32)
    mixed = g.standard_normal((12, E)).astype(np.float32)
    mixed[1::2] = ulps[1::2]
    s = moe.scores(mixed[0].astype(np.float64), score)
    level = (1.5 - s).astype(np.float32)
    copies = np.tile(g.standard_normal((12, E // groups)).astype(np.float32), (1, groups))
    at = g.integers(0, E, 12)
    copies[np.arange(12), at] = np.nextafter(copies[np.arange(12), at], np.float32(9))
    for x, bias in ((ulps, np.full(E, 0.5, np.float32)), (mixed, level), (copies, np.full(E, 0.25, np.float32))):
        t = torch.from_numpy(x).to(dev())
        kw = dict(groups=groups, top_groups=top, group_best=best)
        w, e = mxq.moe_route(t, k, score=score, bias=torch.from_numpy(bias).to(dev()), **kw)
        want_w, want_e = moe.route(f64(t), k, score, bias=bias.astype(np.float64), **kw)
        assert np.array_equal(e.cpu().numpy(), want_e)
        assert_rounded(w, want_w, "f32", 4 * U * want_w, "weights")
