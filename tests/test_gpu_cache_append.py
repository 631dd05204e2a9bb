"""GPU parity of cache_append against the CPU oracle, bit for bit: every format,
block, head size and type; lengths inside and at the ends of pages; padding;
positions without a page, pages that are shared, and everything else left as it
was."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from oracle import paged
from tests.gpu_util import DTYPES, dev
from tests.moe_util import f64
from tests.paged_util import assert_same_pools, counted, on_gpu, pools, table_of, table_on_gpu, values

pytestmark = pytest.mark.gpu


def check(g, cache, table, T, dtype, what, counts=None, make=None):
    heads, dim = cache["k_codes"].shape[1], cache["k_scales"].shape[3] * cache["block"]
    B = len(table[0])
    k, v = (make or values)(g, (B, T, heads, dim), dtype), values(g, (B, T, heads, dim), dtype)
    if cache["v_codes"] is None:
        v = None
    gpu, put = on_gpu(cache), lambda t: None if t is None else t.to(dev())
    mxq.cache_append(gpu, table_on_gpu(table), put(k), put(v),
                     counts=None if counts is None else torch.from_numpy(counts).to(dev()))
    paged.append(cache, table, f64(k), None if v is None else f64(v), counts)
    assert_same_pools(gpu, cache, what)


@pytest.mark.parametrize("fmt,block,dim", [
    ("fp8", 16, 64), ("fp8", 128, 128), ("fp8", 32, 256), ("fp8", 64, 512), ("fp8", 128, 512), ("mxfp4", 32, 64),
    ("mxfp4", 16, 128), ("mxfp4", 128, 256), ("mxfp4", 64, 512), ("nvfp4", 16, 64), ("nvfp4", 16, 512), ("nvfp4", 64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_formats(fmt, block, dim, dtype):
    g = np.random.default_rng(dim + block)
    lengths, T = [0, 13, 16, 31], 5
    cache = pools(g, 14, 3, 16, dim, fmt, block)
    table = counted(table_of(g, [n + T for n in lengths], 16, 3, 14), lengths, 14)
    wide = lambda g, shape, dtype: values(g, shape, dtype) * torch.exp2(  # noqa: E731
        torch.from_numpy(g.integers(-12, 9, shape[:-1] + (1,)).astype(np.float32))).to(DTYPES[dtype])
    check(g, cache, table, T, dtype, f"{fmt}/{block} {dim} {dtype}", np.array([5, 0, 3, 5], np.int32), wide)


@pytest.mark.parametrize("size", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("heads,shared", [(1, False), (8, False), (5, True)])
def test_pages_and_heads(size, heads, shared):
    g = np.random.default_rng(size + heads)
    lengths, T = [size - 1, 2 * size, 7], size + 3
    cache = pools(g, 12, heads, size, 64, "mxfp4", 32, shared)
    table = counted(table_of(g, [n + T for n in lengths], size, 4, 12), lengths, 12)
    check(g, cache, table, T, "bf16", f"pages of {size}")


def test_zeros_of_both_signs_and_the_smallest_values():
    g = np.random.default_rng(0)
    cache = pools(g, 4, 1, 16, 64, "fp8", 32)
    table = counted(np.array([[2]], np.int32), [3], 4)

    def make(g, shape, dtype):
        x = torch.zeros(shape)
        x[0, 0, 0, ::2], x[0, 1], x[0, 2] = -0.0, 2.0 ** -140, -2.0 ** -127
        x[0, 3, 0, 5] = 3e38
        return x
    check(g, cache, table, 4, "f32", "small values", make=make)


def test_places_that_may_not_be_written():
    """No page, a page outside the pool, a shared page, a free page, past the table, lengths out of range."""
    g = np.random.default_rng(1)
    cache = pools(g, 10, 2, 16, 64, "nvfp4", 16)
    rows = np.array([[3, -1, 4], [3, 10, -7], [5, 1 << 30, 6], [7, 8, 9], [0, 1, 2]], np.int32)
    refs = np.array([1, 1, 1, 2, 1, 1, 1, 0, -1, 1], np.int32)
    table = rows, np.array([14, 8, 20, 10, -5], np.int32), refs
    check(g, cache, table, 40, "bf16", "places", np.array([40, 40, 40, 40, 9], np.int32))
    table = rows, np.array([48, 47, 2 ** 31 - 1, 100, -2 ** 31], np.int32), refs
    check(g, cache, table, 3, "bf16", "lengths", np.array([3, 3, 3, 3, -4], np.int32))


def test_prompts_of_many_tokens():
    g = np.random.default_rng(2)
    cache = pools(g, 40, 2, 64, 128, "fp8", 128)
    table = counted(table_of(g, [700, 1100], 64, 18, 40), [0, 17], 40)
    check(g, cache, table, 1083, "bf16", "prompts", np.array([700, 1083], np.int32))


@pytest.mark.parametrize("dim,heads,T", [(64, 9, 1), (64, 200, 1), (128, 5, 2), (512, 33, 1), (512, 3, 15), (256, 2, 70),
                                         (64, 3, 129)])
def test_tiles_that_tokens_and_heads_do_not_fill(dim, heads, T):
    g = np.random.default_rng(dim + heads)
    lengths = [5, 0, 31]
    cache = pools(g, 20, heads, 32, dim, "mxfp4", 16)
    table = counted(table_of(g, [n + T for n in lengths], 32, 6, 20), lengths, 20)
    check(g, cache, table, T, "bf16", f"{heads} heads, {T} tokens", np.array([T, T, T - 1], np.int32))


def test_nothing_to_append():
    g = np.random.default_rng(3)
    cache = pools(g, 4, 2, 16, 64, "fp8", 32)
    table = counted(table_of(g, [16], 16, 1, 4), [0], 4)
    check(g, cache, table, 0, "bf16", "no tokens")
    none = np.zeros((0, 1), np.int32), np.zeros(0, np.int32), np.zeros(4, np.int32)
    check(g, cache, none, 3, "bf16", "no sequences")


def test_strides_and_offsets():
    g = np.random.default_rng(4)
    cache = pools(g, 8, 2, 16, 64, "fp8", 64)
    table = counted(table_of(g, [20, 12], 16, 2, 8), [17, 0], 8)
    k, v = values(g, (2, 2, 3, 64), "bf16"), values(g, (2, 2, 3, 64), "bf16")        # [B, heads, T, D]
    gpu = on_gpu(cache)
    flat = torch.zeros(1 + v.numel(), dtype=torch.bfloat16, device=dev())            # 2 bytes off any alignment
    flat[1:] = v.transpose(1, 2).reshape(-1).to(dev())
    mxq.cache_append(gpu, table_on_gpu(table), k.to(dev()).transpose(1, 2), flat[1:].view(2, 3, 2, 64))
    paged.append(cache, table, f64(k.transpose(1, 2)), f64(v.transpose(1, 2)))
    assert_same_pools(gpu, cache, "strided")


def test_refusals():
    g = np.random.default_rng(5)
    cache = pools(g, 4, 2, 16, 64, "fp8", 32)
    gpu, table = on_gpu(cache), table_on_gpu(counted(np.array([[1]], np.int32), [0], 4))
    k = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16, device=dev())
    with pytest.raises(ValueError):
        mxq.cache_append(gpu, table, k)                                    # no values
    with pytest.raises(ValueError):
        mxq.cache_append(gpu._replace(v_codes=None, v_scales=None), table, k, k)
    with pytest.raises(ValueError):
        mxq.cache_append(gpu, table, k[..., :32], k[..., :32])
    with pytest.raises(ValueError):
        mxq.cache_append(gpu, table, k, k.float())
    with pytest.raises(ValueError):
        mxq.cache_append(gpu, table, k.repeat(2, 1, 1, 1), k.repeat(2, 1, 1, 1))
    with pytest.raises(TypeError):
        mxq.cache_append(gpu, table, k.long(), k.long())
    with pytest.raises(TypeError):
        mxq.cache_append(gpu, table, k, k, counts=torch.ones(1, dtype=torch.int64, device=dev()))
    with pytest.raises(TypeError):
        mxq.cache_append(gpu, table._replace(lengths=table.lengths.long()), k, k)
    with pytest.raises(ValueError):
        mxq.cache_append(gpu, table._replace(refs=table.refs[:3]), k, k)
    with pytest.raises(ValueError, match="contiguous"):
        mxq.cache_append(gpu._replace(k_codes=gpu.k_codes.transpose(1, 2).contiguous().transpose(1, 2)), table, k, k)
    with pytest.raises(ValueError, match="gradient"):
        mxq.cache_append(gpu, table, k.clone().requires_grad_(True), k)
    with pytest.raises(mxq.MxqError):
        mxq.cache_append(gpu._replace(k_codes=gpu.k_codes[:, :, :8].contiguous(), k_scales=gpu.k_scales[:, :, :8].contiguous(),
                                      v_codes=gpu.v_codes[:, :, :8].contiguous(), v_scales=gpu.v_scales[:, :, :8].contiguous()),
                         table, k, k)
    assert_same_pools(gpu, cache, "refused calls")
