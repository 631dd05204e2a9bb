"""The third part of the C ABI (include/mxq_pages.h): the library exports every
entry point, and bad arguments are refused on the host before any HIP call (no
GPU needed)."""

import ctypes
import os
import re

import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from nvfp4_quantization_grouped_amd import _lib
from tests.test_abi_moe import caller

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = [0x10000000 * (i + 1) for i in range(16)]    # disjoint, aligned, never dereferenced
NULL, SHAPE, DTYPE, FORMAT, BLOCK, ALIGN, ALIAS = -1, -2, -3, -4, -5, -6, -7


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libmxq.so is not built (python -m nvfp4_quantization_grouped_amd.build)")
    return _lib.cache_lib()


def cache(**kw):
    fields = dict(pages=64, page_size=32, kv_heads=4, head_dim=128, fmt=0, block=32, k_codes=A[8], k_scales=A[9],
                  v_codes=A[10], v_scales=A[11])
    assert set(kw) <= set(fields)
    return ctypes.byref(_lib.Cache(*{**fields, **kw}.values()))


BAD_CACHES = [
    (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE),
    (dict(page_size=512), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=1025), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(fmt=3), FORMAT), (dict(fmt=-1), FORMAT), (dict(block=8), BLOCK),
    (dict(block=0), BLOCK), (dict(block=256), BLOCK), (dict(head_dim=64, block=128), BLOCK)]
BAD_POOLS = [
    (dict(k_codes=None), NULL), (dict(k_scales=None), NULL), (dict(v_codes=None), NULL), (dict(v_scales=None), NULL),
    (dict(k_codes=A[8] + 8), ALIGN), (dict(v_scales=A[11] + 4), ALIGN)]


def test_header_declares_the_entry_points(L):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxq_pages.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(_lib.CACHE_EXPORTS) == sorted(_lib._CACHE_SIGS)
    for n in names:
        assert isinstance(getattr(L, n), ctypes._CFuncPtr)


def bad_caches(call):
    assert call(cache=None) == NULL
    for kw, status in BAD_CACHES + BAD_POOLS:
        assert call(cache=cache(**kw)) == status, kw


def bad_tables(call):
    for kw in (dict(sequences=-1), dict(sequences=(1 << 20) + 1), dict(width=0), dict(width=(1 << 25) + 1),
               dict(sequences=1 << 12, width=1 << 19)):
        assert call(**kw) == SHAPE, kw


def test_append(L):
    call = caller(L.cache_append, "cache table sequences width lengths refs k v t tokens counts stream",
                  (cache(), A[0], 8, 16, A[1], A[2], A[3], A[4], 1, 2, A[5], None))
    bad_caches(call)
    bad_tables(call)
    assert call(tokens=-1) == call(tokens=(1 << 20) + 1) == call(tokens=1 << 20, sequences=1 << 18) == SHAPE
    assert call(t=3) == DTYPE
    assert call(table=None) == call(lengths=None) == call(refs=None) == call(k=None) == call(v=None) == NULL
    assert call(cache=cache(v_codes=None, v_scales=None)) == NULL          # values for a cache that has none
    assert call(table=A[0] + 1) == call(lengths=A[1] + 2) == call(refs=A[2] + 2) == call(counts=A[5] + 1) == ALIGN
    assert call(k=A[8]) == call(v=A[11] + 16) == call(table=A[9]) == call(refs=A[10]) == call(counts=A[8]) == ALIAS
    assert call(cache=cache(v_codes=A[8] + 32)) == call(cache=cache(k_scales=A[10])) == ALIAS
    assert call(tokens=0) == call(sequences=0) == 0


def test_attention(L):
    W = caller(L.cache_attention_workspace, "cache sequences width t tokens heads", (cache(), 8, 16, 1, 4, 32))
    assert W() >= 0 and W() % 4 == 0 and W(sequences=0) == W(tokens=0) == 0
    for kw, status in BAD_CACHES:
        assert W(cache=cache(**kw)) == status, kw
    assert W(cache=cache(k_codes=None, k_scales=None, v_codes=None, v_scales=None)) == W()
    assert W(t=9) == DTYPE and W(heads=30) == W(heads=0) == W(tokens=1025) == W(width=0) == SHAPE
    call = caller(L.cache_attention, "cache table sequences width lengths q t tokens heads mask each counts scale out lse "
                  "work bytes stream", (cache(), A[0], 8, 16, A[1], A[2], 1, 4, 32, A[3], 1, A[4], 0.1, A[5], A[6], A[7],
                                        1 << 27, None))
    bad_caches(call)
    bad_tables(call)
    assert call(tokens=-1) == call(tokens=1025) == call(heads=30) == call(heads=0) == call(heads=1 << 15) == SHAPE
    assert call(heads=1 << 14, tokens=1024, sequences=1 << 10) == SHAPE
    assert call(t=-1) == DTYPE
    assert call(scale=float("nan")) == call(scale=float("inf")) == call(scale=-2.0 ** 127) == SHAPE
    assert call(table=None) == call(lengths=None) == call(q=None) == call(out=None) == NULL
    assert call(q=A[2] + 8) == call(out=A[5] + 8) == call(lse=A[6] + 2) == call(counts=A[4] + 2) == ALIGN
    assert call(out=A[2] + 64) == call(lse=A[5] + 64) == call(out=A[3]) == call(lse=A[8]) == call(out=A[11]) == ALIAS
    assert call(lse=A[1]) == ALIAS
    if W() > 0:
        assert call(bytes=W() - 1) == SHAPE and call(work=None) == NULL and call(work=A[7] + 4) == ALIGN
        assert call(work=A[5]) == call(work=A[0]) == ALIAS
    assert call(tokens=0) == call(sequences=0) == 0


def test_fork(L):
    call = caller(L.cache_fork, "table sequences width lengths refs pages size parents children keep release table_out "
                  "lengths_out refs_out stream", (A[0], 8, 16, A[1], A[2], 64, 32, A[3], 8, A[4], 1, A[5], A[6], A[7], None))
    bad_tables(call)
    assert call(pages=0) == call(size=24) == call(children=-1) == call(children=1 << 21) == SHAPE
    assert call(parents=None, children=7) == SHAPE
    assert call(table=None) == call(lengths=None) == call(refs=None) == NULL
    assert call(table_out=None) == call(lengths_out=None) == call(refs_out=None) == NULL
    assert call(parents=A[3] + 1) == call(keep=A[4] + 2) == call(refs_out=A[7] + 2) == ALIGN
    assert call(table_out=A[0]) == call(refs_out=A[2]) == call(lengths_out=A[1]) == call(lengths_out=A[5] + 4) == ALIAS
    assert call(table_out=A[3]) == call(refs_out=A[4]) == ALIAS


def test_reserve(L):
    W = L.cache_reserve_workspace
    assert W(-1, 16, 64) == W(4097, 16, 64) == W(8, 0, 64) == W(8, 16, 0) == W(8, 16, 1 << 31) == SHAPE
    assert W(8, 16, 64) > 0 and W(8, 16, 64) % 4 == 0 and W(0, 16, 64) > 0
    call = caller(L.cache_reserve, "cache table sequences width lengths refs tokens each table_out refs_out short work "
                  "bytes stream", (cache(), A[0], 8, 16, A[1], A[2], 1, A[3], A[4], A[5], A[6], A[7], 1 << 20, None))
    bad_caches(call)
    bad_tables(call)
    assert call(sequences=4097) == call(bytes=8) == call(tokens=(1 << 30) + 1) == SHAPE
    assert call(table=None) == call(lengths=None) == call(refs=None) == call(table_out=None) == NULL
    assert call(refs_out=None) == call(short=None) == call(work=None) == NULL
    assert call(each=A[3] + 2) == call(short=A[6] + 1) == call(work=A[7] + 2) == ALIGN
    assert call(table_out=A[0]) == call(refs_out=A[2]) == call(short=A[1]) == call(work=A[3]) == ALIAS
    assert call(refs_out=A[8]) == call(work=A[11]) == call(table=A[9]) == ALIAS


def test_accept(L):
    call = caller(L.cache_accept, "cache table sequences width lengths refs accepted most lengths_out stream",
                  (cache(), A[0], 8, 16, A[1], A[2], A[3], 5, A[4], None))
    bad_caches(call)
    bad_tables(call)
    assert call(most=-1) == call(most=65) == SHAPE
    assert call(table=None) == call(refs=None) == call(accepted=None) == call(lengths_out=None) == NULL
    assert call(accepted=A[3] + 2) == call(lengths_out=A[4] + 2) == ALIGN
    assert call(lengths_out=A[1]) == call(lengths_out=A[3]) == call(accepted=A[8]) == ALIAS
    assert call(sequences=0) == 0


def test_compact(L):
    assert L.cache_compact_workspace(0) == L.cache_compact_workspace(1 << 31) == SHAPE
    assert L.cache_compact_workspace(1) > 0 and L.cache_compact_workspace(63) % 4 == 0
    call = caller(L.cache_compact, "cache table sequences width refs table_out refs_out work bytes stream",
                  (cache(), A[0], 8, 16, A[2], A[4], A[5], A[7], 1 << 20, None))
    bad_caches(call)
    bad_tables(call)
    assert call(bytes=16) == SHAPE
    assert call(table=None) == call(refs=None) == call(table_out=None) == call(refs_out=None) == call(work=None) == NULL
    assert call(work=A[7] + 1) == call(refs=A[2] + 2) == ALIGN
    assert call(table_out=A[0]) == call(refs_out=A[2]) == call(work=A[4]) == call(work=A[8]) == ALIAS


def test_operators_refuse_what_they_cannot_take():
    c = mxq.paged_cache(4, 16, 2, 64, "fp8", 32, device="cpu")
    t = mxq.page_table(3, 2, c)
    assert t.pages.shape == (3, 2) and int(t.pages.max()) == -1 and t.refs.shape == (4,)
    x, n = torch.zeros(3, 1, 2, 64), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: mxq.cache_append(c, t, x, x), lambda: mxq.cache_attention(x, c, t),
                 lambda: mxq.cache_fork(t, n), lambda: mxq.cache_free(c, t), lambda: mxq.cache_reserve(c, t, 1),
                 lambda: mxq.cache_accept(c, t, n[:, None]), lambda: mxq.cache_compact(c, t)):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()
    for kw in (dict(page_size=24), dict(head_dim=80), dict(format="int8"), dict(block_size=8), dict(block_size=128),
               dict(pages=0), dict(kv_heads=0)):
        with pytest.raises(ValueError):
            mxq.paged_cache(**{**dict(pages=4, page_size=16, kv_heads=2, head_dim=64, format="fp8", block_size=32,
                                      device="cpu"), **kw})
    with pytest.raises(ValueError, match="belong together"):
        mxq.cache_compact(c._replace(v_scales=None), t)
    with pytest.raises(ValueError, match="format"):
        mxq.cache_compact(c._replace(format="bf16"), t)
