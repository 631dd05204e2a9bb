"""Helpers of the routed-expert layer's GPU tests: seeded inputs on the device,
float64 views of them for the oracle, and the bounds that results are held to."""

import numpy as np
import torch

from tests.gpu_util import DTYPES, dev

# Half a unit in the last place, relative, and the spacing of the subnormals.
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}
U = 2.0 ** -24           # one fp32 rounding


def values(g, shape, dtype, std=1.0):
    """Normal values of `dtype` on the device."""
    return torch.from_numpy((g.standard_normal(shape) * std).astype(np.float32)).to(DTYPES[dtype]).to(dev())


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def assert_rounded(got, want, dtype, slack, what):
    """|got - want| <= half a step of `dtype` at want, and `slack` (an absolute bound on the arithmetic before the
    rounding; it moves the rounded value by itself and by a half step of its own)."""
    got, want = f64(got), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    slack = np.broadcast_to(np.asarray(slack, np.float64), want.shape)
    bound = HALF[dtype] * (np.abs(want) + slack) + TINY[dtype] + slack
    off = np.abs(got - want)
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; at {i} got {got[i]!r} want {want[i]!r} "
                             f"bound {bound[i]!r}")
