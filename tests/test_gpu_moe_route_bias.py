"""GPU parity of the router under biases far from the scores: experts pinned
with +inf, in each of the three kernels (16 lanes a token, a wave a token, fp64
keys throughout), against the float64 oracle."""

import numpy as np
import pytest

from tests.moe_util import values
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
