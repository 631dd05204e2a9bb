"""Pools without heads, pages or channels are refused by every call that takes them, with the
library's error and before anything runs."""

import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,heads,size,dim", [(4, 0, 16, 64), (0, 2, 16, 64), (4, 2, 0, 64), (4, 2, 16, 0)])
def test_pools_of_nothing(pages, heads, size, dim):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=dev())  # noqa: E731
    cache = mxq.PagedCache(u8(pages, heads, size, dim), u8(pages, heads, size, 2), None, None, "fp8")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev())  # noqa: E731
    table = mxq.PageTable(i32(3, 2), i32(3), i32(pages))
    rows, q = torch.zeros(3, 1, heads, dim, device=dev()), torch.zeros(3, 1, 4, dim, device=dev())
    calls = [lambda: mxq.cache_attention(q, cache, table), lambda: mxq.cache_append(cache, table, rows),
             lambda: mxq.cache_reserve(cache, table, 1), lambda: mxq.cache_accept(cache, table, i32(3, 1)),
             lambda: mxq.cache_compact(cache, table)]
    if pages == 0 or size == 0:              # (which is what cache_free takes of a cache)
        calls.append(lambda: mxq.cache_free(cache, table))
    for call in calls:
        with pytest.raises(mxq.MxqError):
            call()
