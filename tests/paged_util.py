"""Helpers of the paged cache's tests: seeded pools and tables as NumPy arrays
for the oracle and as device tensors for the library, and the bounds that
attention is held to."""

import numpy as np
import torch

import oracle
import nvfp4_quantization_grouped_amd as mxq
from oracle import paged
from tests.gpu_util import DTYPES, dev
from tests.moe_util import U, assert_rounded, f64

# What the probabilities are off by before the products: for bf16 outputs one fp16 part (a half step of 2^-11) or two bf16
# parts, two bf16 parts (two half steps of 2^-8) for fp16, three for fp32.
PARTS = {"bf16": 2.0 ** -11, "f16": 2.0 ** -16, "f32": 2.0 ** -24}
# And of a row's largest: fp16's spacing of 2^-24 below 2^-14, half of it, where the largest is 2^6.
FLOOR = {"bf16": 2.0 ** -31, "f16": 0.0, "f32": 0.0}


def pools(g, pages, heads, size, dim, fmt, block, shared=False, std=1.0):
    """Pools of quantized normal rows."""
    out = dict(fmt=fmt, block=block, k_codes=None, k_scales=None, v_codes=None, v_scales=None)
    for name in ("k",) if shared else ("k", "v"):
        x = g.standard_normal((pages, heads, size, dim)).astype(np.float32).astype(np.float64) * std
        out[name + "_codes"], out[name + "_scales"] = oracle.quantize_cache_packed(x, fmt, block)
    return out


def table_of(g, needs, size, width, pages):
    """Entries for sequences that need so many positions each, in random pages of the pool."""
    order = list(g.permutation(pages))
    rows = np.full((len(needs), width), -1, np.int32)
    for b, n in enumerate(needs):
        for i in range(min(-(-n // size), width)):
            rows[b, i] = order.pop()
    return rows


def counted(rows, lengths, pages):
    return rows, np.asarray(lengths, np.int32), paged._count(rows, pages)


def on_gpu(cache, device=None):
    put = lambda a: None if a is None else torch.from_numpy(a).to(device or dev())  # noqa: E731
    return mxq.PagedCache(*(put(cache[n]) for n in paged.POOLS), cache["fmt"])


def table_on_gpu(table, device=None):
    return mxq.PageTable(*(torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(device or dev()) for a in table))


def copied(cache):
    return {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in cache.items()}


def assert_same_pools(got, want, what):
    for name in paged.POOLS:
        if want[name] is not None:
            a = getattr(got, name).cpu().numpy()
            bad = np.argwhere(a != want[name])
            assert bad.size == 0, f"{what}: {name}: {len(bad)} bytes differ, first at {tuple(bad[0])}"


def assert_same_table(got, want, what):
    for name, a, b in zip(("pages", "lengths", "refs"), got, want):
        a = a.cpu().numpy()
        assert a.shape == b.shape and np.array_equal(a, b), f"{what}: {name}: {np.argwhere(a != b)[:4].tolist()}"


def values(g, shape, dtype, std=1.0):
    return torch.from_numpy((g.standard_normal(shape) * std).astype(np.float32)).to(DTYPES[dtype])


def check_attention(q, cache, table, what, gpu=None, mask=None, counts=None, scale=None, dtype="bf16"):
    """cache_attention on the device against the oracle, within what fp32 sums and the parts of the products allow.

    With a = scale * max sum |q_d k_d|: a score's sum is off by at most D + 2 roundings of a, times log2(e) and the
    running maximum's subtraction 4 more (the exponent's argument is at most a + its maximum, in fp32), which is the
    relative error of each probability; exp2 adds 2 roundings, the parts of p their remainder, the two sums over n
    positions n + 64 roundings each (64: the joining of parts), the division 1.  Relative to the largest one, a
    probability below 2^-126, and what a part below that holds, is 0 in fp32 and bf16: with up to three parts and the
    probability itself 4 * 2^-126 of a value's size for each position (2^-31 where parts are fp16)."""
    c, t = gpu if gpu is not None else (on_gpu(cache), table_on_gpu(table))
    put = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev())  # noqa: E731
    out, lse = mxq.cache_attention(q.to(dev()), c, t, mask=put(mask), counts=put(counts), scale=scale, return_lse=True)
    want, want_lse, reach, mass, peak, met = paged.attention(f64(q), cache, table, mask, counts, scale)
    D = q.shape[-1]
    off = 2 * reach * (D + 6) * U + 2 * U
    rel = 2 * off + PARTS[dtype] + (2 * met + 140) * U
    gone = (4 * 2.0 ** -126 + FLOOR[dtype]) * met[..., None] * peak
    assert_rounded(out, want, dtype, rel[..., None] * mass + gone, f"{what} out")
    got_lse = f64(lse)
    empty = met == 0
    assert np.array_equal(np.isneginf(got_lse), empty), f"{what}: lse of rows with nothing"
    bound = off + (met + 70) * U + U * np.abs(np.where(empty, 0, want_lse)) * 2
    assert (np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, want_lse)) <= bound).all(), f"{what} lse"
    assert not f64(out)[empty].any(), f"{what}: rows with nothing are 0"
    return out, lse
