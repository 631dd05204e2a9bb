"""cache_attention past 2^24 problems (a sequence's kv head each): more than one
row of a launch's grid can hold."""

import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


def test_past_two_to_the_24_problems():
    """2^20 sequences of 17 kv heads each, against the same sequences 2^16 at a time."""
    B, H, D, pages, part = 1 << 20, 17, 64, 40, 1 << 16
    g = torch.Generator(device=dev()).manual_seed(0)
    cache = mxq.paged_cache(pages, 16, H, D, "fp8", 64)
    rows = torch.randn(pages, 16, H, D, generator=g, device=dev())
    whole = mxq.page_table(pages, 1, cache)
    whole = whole._replace(pages=torch.arange(pages, dtype=torch.int32, device=dev())[:, None], refs=whole.refs + 1)
    mxq.cache_append(cache, whole, rows, -rows)
    table = mxq.PageTable(torch.randint(-1, pages, (B, 1), generator=g, device=dev(), dtype=torch.int32),
                          torch.randint(0, 16, (B,), generator=g, device=dev(), dtype=torch.int32),
                          torch.zeros(pages, dtype=torch.int32, device=dev()))
    q = torch.randn(B, 1, H, D, generator=g, device=dev(), dtype=torch.bfloat16)
    out, lse = mxq.cache_attention(q, cache, table, return_lse=True)
    for first in range(0, B, part):
        some = slice(first, first + part)
        want, want_lse = mxq.cache_attention(q[some], cache, mxq.PageTable(table.pages[some], table.lengths[some], table.refs),
                                             return_lse=True)
        assert torch.equal(out[some], want) and torch.equal(lse[some], want_lse), first
    assert bool((out[table.pages[:, 0] < 0] == 0).all()) and bool(out[table.pages[:, 0] >= 0].any(-1).all())
