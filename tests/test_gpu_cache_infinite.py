"""cache_attention over values whose scale times code is past bf16: infinities,
and NaN, of the rows that attend to them, wherever the tile that holds them
ends, however small their probability is, and nothing anywhere else."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from oracle import paged
from tests.gpu_util import dev
from tests.moe_util import f64
from tests.paged_util import copied, counted, on_gpu, pools, table_of, table_on_gpu, values

pytestmark = pytest.mark.gpu


def put(cache, page, kv, row, channel, what):
    """One channel's value +inf, -inf or (fp8) a NaN code; the others of its scale's block 0."""
    fmt, block = cache["fmt"], cache["block"]
    codes, scales = cache["v_codes"][page, kv, row], cache["v_scales"][page, kv, row]
    first = channel // block * block
    if fmt == "fp8":
        codes[first:first + block] = 0
        codes[channel] = {"+": 0x7E, "-": 0xFE, "nan": 0xFF}[what]
    else:
        codes[first // 2:(first + block) // 2] = 0
        codes[channel // 2] = {"+": 0x7, "-": 0xF}[what] << 4 * (channel % 2)
    scales[channel // block] = 250 if fmt == "fp8" else 253


def finite(cache):
    """The same with those codes 0: what every other output has to be."""
    out = copied(cache)
    big = np.repeat(out["v_scales"] >= 240, cache["block"] // (1 if cache["fmt"] == "fp8" else 2), -1)
    out["v_codes"][big] = 0
    return out


def check(q, cache, table, what, mask=None, counts=None, scale=None):
    def run(c):
        on = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev())  # noqa: E731
        return mxq.cache_attention(q.to(dev()), on_gpu(c), table_on_gpu(table), mask=on(mask), counts=on(counts),
                                   scale=scale, return_lse=True)
    with np.errstate(invalid="ignore"):
        want = paged.attention(f64(q), cache, table, mask, counts, scale)[0]
    out, lse = run(cache)
    plain, plain_lse = run(finite(cache))
    got = f64(out)
    odd = ~np.isfinite(want)
    assert odd.any()
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN at {np.argwhere(np.isnan(got) != np.isnan(want))[:5].tolist()}"
    assert np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)]), f"{what}: infinities"
    assert np.array_equal(got[~odd], f64(plain)[~odd]), f"{what}: other outputs"
    assert torch.equal(lse, plain_lse)


KINDS = [("fp8", 32, 64, "bf16"), ("mxfp4", 32, 64, "bf16"), ("fp8", 16, 128, "bf16"), ("mxfp4", 64, 128, "f16"),
         ("fp8", 128, 256, "f32"), ("mxfp4", 16, 512, "bf16"), ("fp8", 64, 512, "bf16"), ("mxfp4", 32, 128, "f32")]


@pytest.mark.parametrize("fmt,block,dim,dtype", KINDS)
@pytest.mark.parametrize("T,heads", [(1, 2), (7, 4), (24, 4)])
def test_infinite_values(fmt, block, dim, dtype, T, heads):
    """In the first tile, in the last one, in drafted rows that some tokens see, in a context that is shared out; one sign,
    both signs, NaN."""
    g = np.random.default_rng(dim + T)
    lengths, size = [75, 0, 33, 1500], 16
    cache = pools(g, sum(-(-(n + T) // size) for n in lengths) + 3, 1, size, dim, fmt, block)
    table = counted(table_of(g, [n + T for n in lengths], size, -(-(1500 + T) // size), len(cache["k_codes"])), lengths,
                    len(cache["k_codes"]))
    q = values(g, (4, T, heads, dim), dtype)
    mask = np.tril(g.random((T, T)) < 0.5) | np.eye(T, dtype=bool)

    def at(b, p, channel, what):
        put(cache, table[0][b, p // size], 0, p % size, channel, what)
    last = dim - 1                         # channels in blocks of their own where there are that many
    at(0, 5, 1, "+")
    at(0, 70, last, "-")
    at(0, 75, 1, "-")                      # token 0 of the draft: both signs for who sees it
    at(2, 31, 1, "+")
    at(2, 32, 1, "+")
    at(3, 3, 1, "+")
    at(3, 1400, last, "-")
    at(3, 700, dim // 2, "+")
    at(3, 900, dim // 2, "-")
    if fmt == "fp8":
        at(3, 1200, dim // 2 - 1, "nan")
    check(q, cache, table, f"{fmt} {dim} {T}", mask)
    check(q, cache, table, f"{fmt} {dim} {T}, padding", mask, counts=np.array([T, T, max(1, T - 2), T - 1], np.int32))


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,heads", [(1, 4), (12, 4)])
def test_the_answer_does_not_depend_on_the_length(fmt, T, heads):
    """The same infinite value in contexts of every length around one tile's end."""
    g = np.random.default_rng(T)
    lengths = list(range(6, 70, 3))
    cache = pools(g, 6 * len(lengths), 1, 16, 64, fmt, 32)
    table = counted(table_of(g, [n + T for n in lengths], 16, 6, len(cache["k_codes"])), lengths, len(cache["k_codes"]))
    for b in range(len(lengths)):
        put(cache, table[0][b, 0], 0, 5, 40, "-")
    q = values(g, (len(lengths), T, heads, 64), "bf16")
    check(q, cache, table, "lengths")
    out = mxq.cache_attention(q.to(dev()), on_gpu(cache), table_on_gpu(table))
    assert torch.isneginf(out[..., 40]).all() and int((~torch.isfinite(out)).sum()) == out[..., 40].numel()


@pytest.mark.parametrize("T,heads,length", [(1, 2, 60), (1, 2, 4000), (20, 2, 60), (20, 2, 4000)])
def test_however_small_the_probability(T, heads, length):
    """Scores far apart: probabilities that fp32 has as 0."""
    g = np.random.default_rng(length + T)
    cache = pools(g, -(-(length + T) // 16) + 1, 1, 16, 64, "mxfp4", 32)
    table = counted(table_of(g, [length + T], 16, -(-(length + T) // 16), len(cache["k_codes"])), [length], len(cache["k_codes"]))
    for p, channel in ((2, 0), (length // 2, 33), (length - 1, 63)):
        put(cache, table[0][0, p // 16], 0, p % 16, channel, "+")
    check(values(g, (1, T, heads, 64), "bf16"), cache, table, "far apart", scale=6.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,heads", [(1, 2), (24, 2)])
def test_large_values_of_no_probability_change_nothing(dtype, T, heads):
    """Values of 2^118 whose probabilities are e^-256, in parts of their own of a context that is shared out: the answer is
    that of the other positions, and what a share of 2^-149 adds is 2^118 * 2^8 * 2048 * 2^-149 = 2^-12 at most."""
    g = np.random.default_rng(T)
    n, size, dim = 4096 - T, 64, 64
    cache = pools(g, 64, 1, size, dim, "fp8", 64)
    table = counted(np.arange(64, dtype=np.int32)[None], [n], 64)
    cache["k_codes"][:32], cache["k_codes"][32:] = 0x38, 0xB8          # 1 and -1
    cache["k_scales"][:] = 127
    cache["v_codes"][:] &= 0x3F                                        # up to 1.875
    cache["v_scales"][:32] = 127
    q = torch.ones(1, T, heads, dim).to(values(g, (1,), dtype).dtype)
    mask = np.zeros((T, T), bool)
    cache["v_scales"][32:] = 127 + 117
    large = paged_run(q, cache, table, mask)
    cache["v_codes"][32:] = 0
    clean = paged_run(q, cache, table, mask)
    assert torch.isfinite(clean).all() and bool((clean > 2.0 ** -10).all())
    assert torch.allclose(large, clean, rtol=2.0 ** -7 if dtype == "bf16" else 2.0 ** -10, atol=2.0 ** -12)


def paged_run(q, cache, table, mask):
    return mxq.cache_attention(q.to(dev()), on_gpu(cache), table_on_gpu(table), mask=torch.from_numpy(mask).to(dev()),
                               scale=2.0).float()
