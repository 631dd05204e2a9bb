"""cache_attention against the float64 oracle: formats, head sizes, groups,
types, lengths from none to many pages, trees, padding, positions without a
page, garbage where nothing is attended to, offsets past 32 bits, streams and
captured graphs.  Bounds: tests/paged_util.py."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from oracle import paged
from tests.gpu_util import DTYPES, dev
from tests.moe_util import f64
from tests.paged_util import (check_attention, copied, counted, on_gpu, pools, table_of, table_on_gpu, values)

pytestmark = pytest.mark.gpu


def tree(g, T, B=None):
    """Each token sees itself and its ancestors."""
    def one():
        m = np.eye(T, dtype=bool)
        for i in range(1, T):
            parent = g.integers(-1, i)
            if parent >= 0:
                m[i] |= m[parent]
        return m
    return one() if B is None else np.stack([one() for _ in range(B)])


def case(g, lengths, T, size, heads, kv_heads, dim, fmt, block, dtype, shared=False, spare=5, std=1.0):
    width = max(1, -(-(max(lengths) + T) // size))
    pages = sum(-(-(n + T) // size) for n in lengths) + spare
    cache = pools(g, pages, kv_heads, size, dim, fmt, block, shared)
    table = counted(table_of(g, [n + T for n in lengths], size, width, pages), lengths, pages)
    return cache, table, values(g, (len(lengths), T, heads, dim), dtype, std)


@pytest.mark.parametrize("fmt,block", [("fp8", 16), ("fp8", 32), ("fp8", 64), ("fp8", 128), ("mxfp4", 16), ("mxfp4", 32),
                                       ("mxfp4", 64), ("mxfp4", 128), ("nvfp4", 16), ("nvfp4", 32), ("nvfp4", 64)])
@pytest.mark.parametrize("dim", [64, 128, 256, 512])
def test_formats(fmt, block, dim):
    if block > dim:
        pytest.skip("a block is no more than a row")
    g = np.random.default_rng(dim + block)
    cache, table, q = case(g, [70, 33, 5], 2, 16, 4, 2, dim, fmt, block, "bf16")
    check_attention(q, cache, table, f"{fmt}/{block} {dim}")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,fmt,block", [(64, "mxfp4", 32), (128, "fp8", 128), (256, "nvfp4", 16), (512, "fp8", 64)])
@pytest.mark.parametrize("shared", [False, True])
def test_types(dtype, dim, fmt, block, shared):
    g = np.random.default_rng(dim)
    cache, table, q = case(g, [40, 0, 129], 3, 32, 6, 2, dim, fmt, block, dtype, shared, std=2.0)
    check_attention(q, cache, table, f"{dtype} {dim}", mask=tree(g, 3, 3), dtype=dtype)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (7, 1), (28, 4), (40, 8), (12, 1), (64, 1), (48, 2)])
@pytest.mark.parametrize("T", [1, 3, 17])
def test_groups(heads, kv_heads, T):
    g = np.random.default_rng(heads + T)
    cache, table, q = case(g, [50, 21], T, 16, heads, kv_heads, 64, "fp8", 32, "bf16")
    check_attention(q, cache, table, f"{heads}/{kv_heads} x {T}")


@pytest.mark.parametrize("size", [16, 32, 64, 128, 256])
def test_lengths_around_pages_and_tiles(size):
    g = np.random.default_rng(size)
    lengths = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500]
    cache, table, q = case(g, lengths, 1, size, 2, 1, 64, "mxfp4", 32, "bf16")
    check_attention(q, cache, table, f"pages of {size}")
    cache, table, q = case(g, lengths, 4, size, 2, 1, 64, "mxfp4", 32, "f16")
    check_attention(q, cache, table, f"pages of {size}, tree", mask=tree(g, 4), dtype="f16")


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "f32"), (256, "bf16"), (512, "f16")])
def test_long_contexts(dim, dtype):
    """Enough positions that the work is split; lengths far apart."""
    g = np.random.default_rng(dim)
    cache, table, q = case(g, [4100, 3, 1777], 2, 64, 4, 1, dim, "nvfp4", 16, dtype, dim == 512)
    check_attention(q, cache, table, f"long {dim}", dtype=dtype)


@pytest.mark.parametrize("T", [2, 16, 33, 64, 130])
def test_trees(T):
    g = np.random.default_rng(T)
    cache, table, q = case(g, [37, 0, 200], T, 32, 4, 2, 64, "fp8", 64, "bf16")
    check_attention(q, cache, table, "one tree", mask=tree(g, T))
    check_attention(q, cache, table, "a tree each", mask=tree(g, T, 3), counts=np.array([T, T - 1, T // 2], np.int32))
    check_attention(q, cache, table, "chains", counts=np.array([1, T, 0], np.int32))


def test_rows_with_nothing():
    g = np.random.default_rng(0)
    cache, table, q = case(g, [0, 0, 9, 40], 5, 16, 4, 2, 64, "fp8", 32, "bf16")
    mask = tree(g, 5, 4)
    mask[0, 2] = False                                   # a token that may not even see itself, and no context
    mask[1] = False
    mask[2, 1] = False                                   # sees its context alone
    check_attention(q, cache, table, "empty masks", mask=mask, counts=np.array([5, 5, 4, -2], np.int32))
    gone = np.full_like(table[0], -1), table[1], table[2]
    check_attention(q, cache, gone, "no pages at all", mask=mask)
    holes = table[0].copy()
    holes[3, 1] = -1                                     # the middle of a context
    holes[2, 0] = len(table[2])                          # outside the pool: the context, and some of the drafts
    check_attention(q, cache, (holes, table[1], table[2]), "holes", mask=mask)


def test_lengths_out_of_range():
    g = np.random.default_rng(1)
    cache, table, q = case(g, [30, 30, 30, 30], 2, 16, 2, 1, 64, "nvfp4", 16, "bf16")
    odd = np.array([-7, 2 ** 31 - 1, 32, 31], np.int32)  # the table ends at 32
    check_attention(q, cache, (table[0], odd, table[2]), "lengths", counts=np.array([2 ** 31 - 1, 2, -2 ** 31, 2], np.int32))


@pytest.mark.parametrize("fmt,block", [("fp8", 32), ("mxfp4", 32), ("nvfp4", 16)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_garbage_that_nothing_attends_to(fmt, block, dtype):
    """NaN codes and scales behind the last position, in other pages, and in drafted rows that some tokens do not see;
    NaN and infinities in padded rows of q."""
    g = np.random.default_rng(2)
    T = 6
    cache, table, q = case(g, [37, 0, 20], T, 16, 4, 2, 64, fmt, block, dtype)
    counts = np.array([6, 6, 4], np.int32)
    mask = np.stack([np.eye(T, dtype=bool)] * 3)
    mask[:, 4, 1] = True
    bad = copied(cache)
    live = np.zeros(cache["k_codes"].shape[:1] + cache["k_codes"].shape[2:3], bool)
    for b, n in enumerate(table[1]):
        for p in range(n + counts[b]):
            live[table[0][b, p // 16], p % 16] = True
    for name in paged.POOLS:
        bad[name].transpose(0, 2, 1, 3)[~live] = 0xFF            # NaN scales (and NaN fp8 codes)
    # drafted token 3 of every sequence, which only token 3 sees: its own output is NaN
    nan = []
    for b, n in enumerate(table[1]):
        p = n + 3
        for name in ("k_scales", "v_scales"):
            bad[name][table[0][b, p // 16], :, p % 16] = 0x7F if fmt == "nvfp4" else 0xFF
        nan.append((b, 3))
    q[2, 4:] = float("nan")
    q[2, 5, 0, 0] = float("inf")
    put = lambda a: torch.from_numpy(a).to(dev())  # noqa: E731
    out, lse = mxq.cache_attention(q.to(dev()), on_gpu(bad), table_on_gpu(table), mask=put(mask), counts=put(counts),
                                   return_lse=True)
    for b, i in nan:
        assert torch.isnan(out[b, i]).all() and torch.isnan(lse[b, i]).all()
    ref, ref_lse = mxq.cache_attention(q.to(dev()), on_gpu(cache), table_on_gpu(table), mask=put(mask),
                                       counts=put(counts), return_lse=True)
    keep = torch.ones(3, T, dtype=torch.bool)
    keep[:, 3] = False
    assert torch.equal(out[keep.to(dev())], ref[keep.to(dev())]) and torch.equal(lse[keep.to(dev())], ref_lse[keep.to(dev())])
    clean = q.clone()
    clean[2, 4:] = 0
    check_attention(clean, cache, table, "the same, clean", mask=mask, counts=counts, dtype=dtype)


def test_nan_of_one_channel_of_a_value_stays_there():
    """An fp8 NaN in one channel of a drafted value: NaN in that channel of the rows that see it, and nowhere else."""
    g = np.random.default_rng(3)
    cache, table, q = case(g, [40, 3], 5, 16, 4, 1, 128, "fp8", 32, "bf16")
    mask = np.eye(5, dtype=bool)
    mask[4, 2] = True
    clean = mxq.cache_attention(q.to(dev()), on_gpu(cache), table_on_gpu(table), mask=torch.from_numpy(mask).to(dev()))
    for b, n in enumerate(table[1]):
        cache["v_codes"][table[0][b, (n + 2) // 16], 0, (n + 2) % 16, 77] = 0x7F
    out = mxq.cache_attention(q.to(dev()), on_gpu(cache), table_on_gpu(table), mask=torch.from_numpy(mask).to(dev()))
    want = torch.zeros_like(clean, dtype=torch.bool)
    want[:, [2, 4], :, 77] = True
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], clean[~want])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nvfp4_scales_with_mantissas(dtype):
    """quantize_cache_packed writes powers of two; any finite E4M3 scale byte means its value."""
    g = np.random.default_rng(4)
    cache, table, q = case(g, [90, 31], 2, 16, 4, 2, 128, "nvfp4", 16, dtype)
    for name in ("k_scales", "v_scales"):
        cache[name] = g.integers(0, 0x50, cache[name].shape).astype(np.uint8)     # up to 16
    check_attention(q, cache, table, "mantissas", dtype=dtype)
    one = copied(cache)
    for name in ("k_scales", "v_scales"):
        one[name][:] = 0x38
        one[name][table[0][0, 2], 1, 5] = 0x3B                                    # one row of one head
    check_attention(q, one, table, "one row's mantissas", dtype=dtype)


def test_scales_far_from_one():
    """Scores near 1e4 and values near 2^100; the largest score late, and early."""
    g = np.random.default_rng(5)
    cache, table, q = case(g, [300, 300], 1, 32, 2, 1, 64, "mxfp4", 32, "f32")
    cache["v_scales"][:] += 100
    cache["k_scales"][table[0][0, 9]] += 6
    cache["k_scales"][table[0][1, 0]] += 6
    check_attention(q, cache, table, "far", dtype="f32", scale=3.0)
    check_attention(q, cache, table, "negative", dtype="f32", scale=-0.5)
    check_attention(q, cache, table, "none", dtype="f32", scale=0.0)


def test_every_code_as_key_and_value():
    g = np.random.default_rng(6)
    for fmt, block in (("fp8", 16), ("mxfp4", 16), ("nvfp4", 16)):
        cache, table, q = case(g, [256], 1, 32, 1, 1, 64, fmt, block, "f32")
        for name in ("k_codes", "v_codes"):
            codes = g.permutation(cache[name].size) % 256
            if fmt == "fp8":
                codes[(codes & 0x7F) == 0x7F] = 0
            cache[name] = codes.astype(np.uint8).reshape(cache[name].shape)
        check_attention(q, cache, table, f"codes of {fmt}", dtype="f32", scale=1e-3)


def test_offsets_past_32_bits():
    """A pool of 4.8 GB whose last pages hold the sequence."""
    pages, size, dim = 9300, 256, 512
    gpu = mxq.paged_cache(pages, size, 4, dim, "fp8", 128, shared=True)
    assert gpu.k_codes.numel() > 1 << 32
    g = np.random.default_rng(7)
    small = pools(g, 4, 4, size, dim, "fp8", 128, True)
    rows = np.array([[0, 1], [2, 3]], np.int32)
    table = counted(rows, [300, 511], 4)
    far = torch.tensor([pages - 1, 8200, 8300, pages - 2], device=dev())
    gpu.k_codes[far] = torch.from_numpy(small["k_codes"]).to(dev())
    gpu.k_scales[far] = torch.from_numpy(small["k_scales"]).to(dev())
    q = values(g, (2, 1, 8, dim), "bf16")
    at = mxq.PageTable(far[torch.from_numpy(rows).to(dev()).long()].to(torch.int32), table_on_gpu(table).lengths,
                       torch.zeros(pages, dtype=torch.int32, device=dev()))
    check_attention(q, small, table, "far pages", gpu=(gpu, at))


def test_strided_and_unaligned_q():
    g = np.random.default_rng(8)
    cache, table, q = case(g, [50, 9], 3, 16, 4, 2, 64, "fp8", 32, "bf16")
    want = mxq.cache_attention(q.to(dev()), on_gpu(cache), table_on_gpu(table))
    turned = q.to(dev()).transpose(1, 2).contiguous().transpose(1, 2)
    flat = torch.zeros(1 + q.numel(), dtype=torch.bfloat16, device=dev())
    flat[1:] = q.reshape(-1).to(dev())
    for other in (turned, flat[1:].view(q.shape)):
        assert torch.equal(mxq.cache_attention(other, on_gpu(cache), table_on_gpu(table)), want)


def test_the_same_answer_every_time():
    g = np.random.default_rng(9)
    cache, table, q = case(g, [3000, 100, 900], 4, 16, 8, 2, 128, "mxfp4", 32, "bf16")
    c, t, x = on_gpu(cache), table_on_gpu(table), q.to(dev())
    first = mxq.cache_attention(x, c, t)
    for _ in range(20):
        assert torch.equal(mxq.cache_attention(x, c, t), first)


def shifted(cache, name, pages, by):
    """The scale exponents of these pages raised (no byte is 255, which is NaN)."""
    x = cache[name][pages].astype(np.int64) + by
    cache[name][pages] = np.clip(x, 0, 254).astype(np.uint8)


@pytest.mark.parametrize("fmt,block", [("fp8", 32), ("fp8", 128), ("mxfp4", 32)])
@pytest.mark.parametrize("dim,T,heads", [(64, 12, 4), (64, 33, 4), (128, 24, 2), (128, 10, 8), (256, 9, 4)])
def test_values_that_fp16_does_not_hold(fmt, block, dim, T, heads):
    """More rows than one tile of 32, whose probabilities are fp16 where the values' scales allow it: values near 2^30,
    near 2^-60 and 0 (scale bytes of 0 as well), in all pages, in one page of a long context, in the drafted rows alone."""
    if block > dim:
        pytest.skip("a block is no more than a row")
    g = np.random.default_rng(dim + T)
    cache, table, q = case(g, [700, 33, 0], T, 16, heads, 1, dim, fmt, block, "bf16")
    mask = tree(g, T)
    used = table[0][table[0] >= 0]
    for what, pages, by in (("all large", used, 30), ("all small", used, -60), ("one page large", table[0][0, 20:21], 18),
                            ("one page small", table[0][0, 3:4], -40), ("drafted", table[0][0, 43:44], 20),
                            ("zero scales", table[0][0, 7:9], -255)):
        other = copied(cache)
        shifted(other, "v_scales", pages, by)
        check_attention(q, other, table, f"{fmt} {what}", mask=mask)
    zero = copied(cache)
    zero["v_codes"][table[0][0, 5]] = 0
    zero["v_scales"][table[0][0, 5]] = 0
    check_attention(q, zero, table, f"{fmt} rows of zeros", mask=mask)


@pytest.mark.parametrize("fmt,block", [("fp8", 32), ("mxfp4", 32), ("nvfp4", 16)])
@pytest.mark.parametrize("dim,T,heads", [(64, 20, 2), (64, 40, 4), (128, 12, 4), (128, 40, 4), (256, 10, 4), (512, 24, 4)])
def test_nan_values_of_many_rows(fmt, block, dim, T, heads):
    """As above where the rows are more than a wave's: a drafted value that is not finite in some channels reaches those
    channels of the rows that see it alone; the first sequence's context is long enough to be shared out."""
    g = np.random.default_rng(dim + T + 1)
    cache, table, q = case(g, [900, 0, 30], T, 16, heads, 1, dim, fmt, block, "bf16")
    mask = np.eye(T, dtype=bool)
    mask[T - 1, [2, 5]] = True
    mask[7, 2] = True
    put = lambda a: torch.from_numpy(a).to(dev())  # noqa: E731
    clean = mxq.cache_attention(q.to(dev()), on_gpu(cache), table_on_gpu(table), mask=put(mask))
    want = torch.zeros_like(clean, dtype=torch.bool)
    for b, n in enumerate(table[1]):
        for token, channel in ((2, dim - 3), (5, 17)):
            page, row = table[0][b, (n + token) // 16], (n + token) % 16
            sees = np.flatnonzero(mask[:, token])
            if fmt == "fp8":
                cache["v_codes"][page, 0, row, channel] = 0xFF
                want[b, sees, :, channel] = True
            else:
                first = channel // block * block
                cache["v_scales"][page, 0, row, channel // block] = 0x7F if fmt == "nvfp4" else 0xFF
                want[b, sees, :, first: first + block] = True
    out = mxq.cache_attention(q.to(dev()), on_gpu(cache), table_on_gpu(table), mask=put(mask))
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], clean[~want])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,T", [(64, 30), (128, 12), (512, 17)])
def test_nvfp4_scales_with_mantissas_of_many_rows(dtype, dim, T):
    g = np.random.default_rng(16)
    cache, table, q = case(g, [300, 31], T, 16, 4, 1, dim, "nvfp4", 16, dtype)
    for name in ("k_scales", "v_scales"):
        x = g.integers(0, 0x40, cache[name].shape)                                # up to 2, of both signs
        cache[name] = (x | g.integers(0, 2, x.shape) << 7).astype(np.uint8)
    check_attention(q, cache, table, "mantissas", mask=tree(g, T), dtype=dtype)


@pytest.mark.parametrize("scale", [1e-6, 40.0])
@pytest.mark.parametrize("T", [1, 20])
def test_probabilities_all_alike_and_of_one_position(scale, T):
    """Scores so close that every position counts, and so far apart that one does, its score first or last."""
    g = np.random.default_rng(17)
    cache, table, q = case(g, [1500, 200], T, 32, 4, 1, 128, "nvfp4", 16, "bf16")
    check_attention(q, cache, table, "scores", scale=scale)


def test_largest_scores_rise_all_the_way():
    """Each tile's largest score is past the last one's by more than the running maximum lets pass."""
    g = np.random.default_rng(18)
    for T in (1, 20):
        cache, table, q = case(g, [640, 640], T, 32, 4, 1, 64, "fp8", 64, "bf16")
        q = q.abs()
        codes, scales = cache["k_codes"], cache["k_scales"]
        codes &= 0x7F                                                   # positive scores
        for b in range(2):
            order = table[0][b] if b == 0 else table[0][b][::-1]
            for i, page in enumerate(p for p in order if p >= 0):
                scales[page] = 118 + min(i, 12)
        check_attention(q, cache, table, f"rising, {T}", scale=1.0)


@pytest.mark.parametrize("B,T,heads,dim", [(65, 1, 4, 64), (300, 1, 4, 64), (300, 10, 4, 64), (130, 17, 2, 128), (520, 2, 2, 64)])
def test_many_sequences_share_the_workgroups(B, T, heads, dim):
    """More sequences than a workgroup has threads, lengths from none to many steps, some of them padding alone."""
    g = np.random.default_rng(B + T)
    lengths = (g.integers(0, 40, B) * g.integers(0, 40, B)).tolist()
    cache, table, q = case(g, lengths, T, 64, heads, 1, dim, "mxfp4", 32, "bf16")
    counts = g.integers(-1, T + 1, B).astype(np.int32)
    counts[g.random(B) < 0.5] = T
    check_attention(q, cache, table, "sequences", counts=counts)


def test_many_long_sequences_of_one_token():
    """The same for a kernel whose waves share the rows, and contexts long enough for it."""
    g = np.random.default_rng(21)
    lengths = (g.integers(0, 61, 300) * g.integers(0, 101, 300)).tolist()
    lengths[0], lengths[299] = 6000, 0
    cache, table, q = case(g, lengths, 1, 64, 4, 1, 64, "mxfp4", 32, "bf16")
    counts = g.integers(0, 2, 300).astype(np.int32)
    counts[:100] = 1
    check_attention(q, cache, table, "sequences", counts=counts)


def test_two_calls_at_once():
    """Two streams, a call of its own on each, over and over: neither sees the other's workspace."""
    g = np.random.default_rng(19)
    made = []
    for fmt, block, T in (("fp8", 32, 1), ("nvfp4", 16, 20)):
        cache, table, q = case(g, [3000, 500, 90], T, 64, 8, 2, 128, fmt, block, "bf16")
        made.append((on_gpu(cache), table_on_gpu(table), q.to(dev()), torch.cuda.Stream()))
    want = [mxq.cache_attention(q, c, t) for c, t, q, _ in made]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, (c, t, q, stream) in enumerate(made):
            with torch.cuda.stream(stream):
                got[i].append(mxq.cache_attention(q, c, t))
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


def test_nothing_to_attend_with():
    g = np.random.default_rng(20)
    cache, table, q = case(g, [20], 2, 16, 4, 2, 64, "fp8", 32, "bf16")
    c = on_gpu(cache)
    out, lse = mxq.cache_attention(torch.empty(0, 3, 4, 64, device=dev()), c, mxq.page_table(0, 2, c), return_lse=True)
    assert out.shape == (0, 3, 4, 64) and lse.shape == (0, 3, 4)
    out, lse = mxq.cache_attention(q.to(dev()), c, table_on_gpu(table), counts=torch.zeros(1, dtype=torch.int32, device=dev()),
                                   return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()


def test_many_short_sequences():
    g = np.random.default_rng(10)
    lengths = list(g.integers(0, 40, 700))
    cache, table, q = case(g, lengths, 1, 16, 2, 1, 64, "fp8", 64, "bf16")
    check_attention(q, cache, table, "many")


def test_refusals():
    g = np.random.default_rng(11)
    cache, table, q = case(g, [20], 2, 16, 4, 2, 64, "fp8", 32, "bf16")
    c, t, x = on_gpu(cache), table_on_gpu(table), q.to(dev())
    eye = torch.eye(2, dtype=torch.bool, device=dev())
    for call, error in (
            (lambda: mxq.cache_attention(x[:, :, :3], c, t), ValueError),
            (lambda: mxq.cache_attention(x[:, :, :0], c, t), ValueError),
            (lambda: mxq.cache_attention(x[..., :32], c, t), ValueError),
            (lambda: mxq.cache_attention(x[0], c, t), ValueError),
            (lambda: mxq.cache_attention(x.repeat(2, 1, 1, 1), c, t), ValueError),
            (lambda: mxq.cache_attention(x.double(), c, t), TypeError),
            (lambda: mxq.cache_attention(x, c, t, mask=eye.float()), TypeError),
            (lambda: mxq.cache_attention(x, c, t, mask=eye[:1]), TypeError),
            (lambda: mxq.cache_attention(x, c, t, mask=eye.cpu()), ValueError),
            (lambda: mxq.cache_attention(x, c, t, counts=torch.ones(2, dtype=torch.int32, device=dev())), TypeError),
            (lambda: mxq.cache_attention(x.repeat(1, 600, 1, 1), c, t), mxq.MxqError),
            (lambda: mxq.cache_attention(x.clone().requires_grad_(True), c, t), ValueError),
            (lambda: mxq.cache_attention(x, c._replace(k_codes=c.k_codes.int()), t), TypeError)):
        with pytest.raises(error):
            call()
    assert mxq.cache_attention(x[:, :0], c, t).shape == (1, 0, 4, 64)
    with torch.no_grad():
        mxq.cache_attention(x.clone().requires_grad_(True), c, t)


def test_another_stream():
    g = np.random.default_rng(12)
    cache, table, q = case(g, [2000, 77], 2, 16, 4, 2, 128, "fp8", 128, "bf16")
    c, t, x = on_gpu(cache), table_on_gpu(table), q.to(dev())
    want = mxq.cache_attention(x, c, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mxq.cache_attention(x, c, t)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_two_captured_steps_replayed_in_turn():
    """Two graphs, each a whole step (reserve, append, attention, accept) over a cache of its own, replayed in turn with
    eager calls between; every replay gives what the eager step gives."""
    g = np.random.default_rng(13)
    T, made = 3, []
    for fmt, block in (("fp8", 32), ("mxfp4", 32)):
        cache, table, q = case(g, [600, 41], T, 16, 4, 2, 64, fmt, block, "bf16", spare=20)
        rows = table[0].copy()
        for b, n in enumerate(table[1]):
            rows[b, -(-n // 16):] = -1
        table = counted(rows, table[1], len(table[2]))
        k, v = values(g, (2, T, 2, 64), "bf16").to(dev()), values(g, (2, T, 2, 64), "bf16").to(dev())
        accepted = torch.tensor([[0, 2], [1, -1]], dtype=torch.int32, device=dev())
        mask = torch.from_numpy(tree(g, T)).to(dev())

        def step(c, t, x, k=k, v=v, accepted=accepted, mask=mask):
            t, short = mxq.cache_reserve(c, t, T)
            mxq.cache_append(c, t, k, v)
            out = mxq.cache_attention(x, c, t, mask=mask)
            return out, mxq.cache_accept(c, t, accepted), short
        static = on_gpu(cache), table_on_gpu(table), q.to(dev())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(on_gpu(cache), *static[1:])
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*static)
        made.append((cache, q, step, static, graph, outs))
    for turn in range(4):
        for cache, q, step, static, graph, outs in made:
            x = torch.randn(q.shape, device=dev()).to(DTYPES["bf16"])
            for name, pool in zip(paged.POOLS, static[0]):
                pool.copy_(torch.from_numpy(cache[name]))
            static[2].copy_(x)
            graph.replay()
            fresh = on_gpu(cache)
            want, after, short = step(fresh, static[1], x)
            torch.cuda.synchronize()
            assert torch.equal(outs[0], want), turn
            assert all(torch.equal(a, b) for a, b in zip(outs[1], after)) and torch.equal(outs[2], short)
            assert all(torch.equal(a, b) for a, b in zip(static[0][:4], fresh[:4]))


def test_a_step_of_drafting_and_a_step_of_beams():
    """The operators together, as a serving loop calls them, against the oracle: a tree drafted, attended to and
    accepted in part, then beams forked, reserved, appended and attended to, then pages freed and compacted."""
    g = np.random.default_rng(14)
    size, dim, T = 16, 128, 6
    cache = pools(g, 60, 2, size, dim, "nvfp4", 16)
    table = counted(table_of(g, [45, 16, 3], size, 8, 60), [45, 16, 3], 60)
    gpu, at = on_gpu(cache), table_on_gpu(table)
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev())  # noqa: E731

    def same(what):
        for a, b in zip(at, table):
            assert np.array_equal(a.cpu().numpy(), b), what
        for name in paged.POOLS:
            assert np.array_equal(getattr(gpu, name).cpu().numpy(), cache[name]), (what, name)

    def write(n):
        k, v = values(g, (len(table[0]), n, 2, dim), "bf16"), values(g, (len(table[0]), n, 2, dim), "bf16")
        mxq.cache_append(gpu, at, k.to(dev()), v.to(dev()))
        paged.append(cache, table, f64(k), f64(v))

    at, _ = mxq.cache_reserve(gpu, at, T)
    table, _ = paged.reserve(cache, table, [T] * 3)
    write(T)
    same("drafted")
    check_attention(values(g, (3, T, 8, dim), "bf16"), cache, table, "drafted", (gpu, at), mask=tree(g, T, 3))
    accepted = np.array([[0, 3, 5], [1, -1, -1], [0, 1, 2]], np.int32)
    at, table = mxq.cache_accept(gpu, at, put(accepted)), paged.accept(cache, table, accepted)
    same("accepted")
    parents = np.array([0, 0, 2, 2, 2], np.int32)
    at, table = mxq.cache_fork(at, put(parents), release=True), paged.fork(table, parents, size, True)
    at, short = mxq.cache_reserve(gpu, at, 1)
    table, lack = paged.reserve(cache, table, [1] * 5)
    assert short.tolist() == lack.tolist() == [0] * 5
    write(1)
    same("beams")
    check_attention(values(g, (5, 1, 8, dim), "bf16"), cache, table, "beams", (gpu, at))
    at = at._replace(lengths=at.lengths + 1)
    table = table[0], table[1] + 1, table[2]
    keep = np.array([99, 0, 4, 99, 0], np.int32)
    at, table = mxq.cache_free(gpu, at, put(keep)), paged.fork(table, range(5), size, True, keep)
    same("freed")
    at, table = mxq.cache_compact(gpu, at), paged.compact(cache, table)
    same("compacted")
    check_attention(values(g, (5, 1, 8, dim), "bf16"), cache, table, "compacted", (gpu, at))
