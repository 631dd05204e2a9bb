"""Every kernel of cache_attention at least once, by itself and shared out with
its join: each type of q, format, head size and number of rows that a tile is
made for."""

import numpy as np
import pytest

from tests.paged_util import check_attention, counted, pools, table_of, values
from tests.test_gpu_cache_attention import tree

pytestmark = pytest.mark.gpu

# (head size, drafted tokens): 4 heads to each, so 4 T rows, in tiles of 16, 32, 64 and 128; two tiles where they are 132
SHAPES = [(dim, T) for dim in (64, 128) for T in (3, 7, 13, 25, 33)] + [(dim, T) for dim in (256, 512) for T in (3, 10, 17)]
FORMATS = [("fp8", 32), ("mxfp4", 64), ("nvfp4", 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,block", FORMATS)
@pytest.mark.parametrize("dim,T", SHAPES)
@pytest.mark.parametrize("shared_out", [False, True])
def test_each_kernel(dtype, fmt, block, dim, T, shared_out):
    g = np.random.default_rng(dim + T)
    # past 14 steps of 128 positions up to 32 rows, past 4 of at most 128 from there on: shared out
    lengths = [90, 17] if not shared_out else [2000, 70] if 4 * T <= (32 if dim <= 128 else 16) else [700, 70]
    size = 32
    pages = sum(-(-(n + T) // size) for n in lengths) + 2
    cache = pools(g, pages, 1, size, dim, fmt, block)
    table = counted(table_of(g, [n + T for n in lengths], size, -(-(max(lengths) + T) // size), pages), lengths, pages)
    counts = np.array([T, T - 1], np.int32)
    check_attention(values(g, (2, T, 4, dim), dtype), cache, table, f"{dtype} {fmt} {dim} x {4 * T}", mask=tree(g, T, 2),
                    counts=counts, dtype=dtype)
