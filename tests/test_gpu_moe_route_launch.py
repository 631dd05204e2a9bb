"""Calls of the router near the limits of one launch."""

import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


def test_route_of_more_tokens_than_a_wave_each_would_launch():
    """Past 2^26 tokens 64 lanes a token are more threads than a launch takes; 16 are not."""
    T = 2 ** 26 + 3
    x = torch.randn(T, 2, device=dev(), dtype=torch.bfloat16, generator=torch.Generator(dev()).manual_seed(3))
    w, e = mxq.moe_route(x, 1)
    assert torch.equal(e[:, 0] == 1, x[:, 1] > x[:, 0]) and (w == 1).all()
