"""A KV cache held packed and in pages: rows quantized into it, attention over
it for one new token or a tree of drafted ones, and its pages.

Argument marshalling only: every step runs in the HIP kernels behind the C ABI
(``include/mxq_pages.h``, which defines each operation).  Tensors must be CUDA
(ROCm) tensors on one device; calls are enqueued on the current stream of that
device, outputs and workspaces are allocated with PyTorch's caching allocator.
There is no CPU path, and no gradient: a tensor that wants one is refused.

Nothing is read back to the host, so everything can be captured into a graph.
The pools are written in place; what a call changes of a table comes back as
new tensors (the rest are the ones that were given), which a loop around a
captured graph copies into the ones it started from.

A step of a serving loop with drafted tokens::

    table, short = cache_reserve(cache, table, tokens)          # short > 0: the pool ran out
    cache_append(cache, table, k, v)                            # rows of this layer
    out = cache_attention(q, cache, table, mask=tree)
    table = cache_accept(cache, table, accepted)                # the path that was verified

and of beam search::

    table = cache_fork(table, parents, release=True)            # beams continue from their parents
    table, short = cache_reserve(cache, table, 1)               # shared last pages become their own

Layers share a table: reserve, fork and free it once a step, with a cache whose
pools hold all layers' heads, or move rows (``cache_reserve``, ``cache_accept``,
``cache_compact``) in each layer's cache with the same table and counts.
"""

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import _lib
from .moe import _differentiated, _float_type, _ptr
from .ops import _FMT, _need_cuda

_PAGE_SIZES = (16, 32, 64, 128, 256)
_HEAD_DIMS = (64, 128, 256, 512)


class PagedCache(NamedTuple):
    """Pools of a packed cache, all uint8 and contiguous.

    k_codes: [pages, kv_heads, page_size, head_dim] (fp8) or [..., head_dim / 2]
        (mxfp4, nvfp4), as ``quantize_cache_packed`` writes rows.
    k_scales: [pages, kv_heads, page_size, head_dim / block_size].
    v_codes, v_scales: the same for the values, or None: the values are the keys.
    format: "fp8", "mxfp4" or "nvfp4".
    """
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: Optional[torch.Tensor]
    v_scales: Optional[torch.Tensor]
    format: str


class PageTable(NamedTuple):
    """Which pages hold which positions.

    pages: int32 [sequences, width], the page of positions i * page_size on; -1 for none.
    lengths: int32 [sequences], cached positions.
    refs: int32 [pages of the pool], how many entries name a page; 0 for a free one.
    """
    pages: torch.Tensor
    lengths: torch.Tensor
    refs: torch.Tensor


def paged_cache(pages, page_size, kv_heads, head_dim, format, block_size, *, shared=False, device="cuda"):
    """Empty pools.  ``page_size`` 16, 32, 64, 128 or 256 positions; ``head_dim``
    64, 128, 256 or 512; ``block_size`` channels share a scale (16, 32, 64 or
    128, no more than head_dim).  With ``shared`` the values are the keys."""
    if format not in _FMT:
        raise ValueError("paged_cache: format must be 'fp8', 'mxfp4' or 'nvfp4'")
    pages, page_size, kv_heads, head_dim, block = (int(n) for n in (pages, page_size, kv_heads, head_dim, block_size))
    if page_size not in _PAGE_SIZES or head_dim not in _HEAD_DIMS or pages < 1 or kv_heads < 1:
        raise ValueError("paged_cache: page_size must be 16, 32, 64, 128 or 256 and head_dim 64, 128, 256 or 512")
    if block not in (16, 32, 64, 128) or block > head_dim:
        raise ValueError("paged_cache: block_size must be 16, 32, 64 or 128 and no more than head_dim")
    rows, pools = (pages, kv_heads, page_size), []
    for width in (head_dim if format == "fp8" else head_dim // 2, head_dim // block) * (1 if shared else 2):
        pools.append(torch.zeros(*rows, width, dtype=torch.uint8, device=device))
    return PagedCache(*pools, *([None, None] if shared else []), format)


def page_table(sequences, width, cache):
    """The table of ``sequences`` empty sequences, of up to ``width`` pages each of ``cache``."""
    device = cache.k_codes.device
    return PageTable(torch.full((int(sequences), int(width)), -1, dtype=torch.int32, device=device),
                     torch.zeros(int(sequences), dtype=torch.int32, device=device),
                     torch.zeros(cache.k_codes.shape[0], dtype=torch.int32, device=device))


def _cache_args(cache, name):
    """The cache as the C ABI takes it, and its device."""
    kc, ks, vc, vs, form = cache
    fmt = _FMT.get(form)
    if fmt is None:
        raise ValueError(f"{name}: format must be 'fp8', 'mxfp4' or 'nvfp4'")
    if (vc is None) != (vs is None):
        raise ValueError(f"{name}: v_codes and v_scales belong together")
    device, index = kc.device, kc.get_device()
    for pool in (kc, ks) if vc is None else (kc, ks, vc, vs):
        if index < 0 or pool.get_device() != index:
            _need_cuda(kc, pool)
            raise ValueError("all tensors must be on the same device")
        if pool.dtype is not torch.uint8 or pool.dim() != 4:
            raise TypeError(f"{name}: pools must be uint8 [pages, kv_heads, page_size, width]")
        if not pool.is_contiguous():
            raise ValueError(f"{name}: pools must be contiguous")
    codes, scales = kc.shape, ks.shape
    pages, heads, size, width = codes
    groups = scales[3]
    dim = width if form == "fp8" else 2 * width
    if scales[0] != pages or scales[1] != heads or scales[2] != size or groups == 0 or dim % groups or (
            vc is not None and (vc.shape != codes or vs.shape != scales)):
        raise ValueError(f"{name}: pools of different shapes")
    return _lib.Cache(pages, size, heads, dim, fmt, dim // groups, kc.data_ptr(), ks.data_ptr(),
                      0 if vc is None else vc.data_ptr(), 0 if vs is None else vs.data_ptr()), device


def _table_args(table, pages, device, name):
    """The table's tensors, contiguous."""
    rows, lengths, refs = table
    if (rows.dtype is not torch.int32 or lengths.dtype is not torch.int32 or refs.dtype is not torch.int32
            or rows.dim() != 2 or lengths.dim() != 1 or refs.dim() != 1):
        raise TypeError(f"{name}: the table must be int32 pages [sequences, width], lengths [sequences] and refs [pages]")
    index = device.index
    if rows.get_device() != index or lengths.get_device() != index or refs.get_device() != index:
        raise ValueError("all tensors must be on the same device")
    if lengths.shape[0] != rows.shape[0] or (pages is not None and refs.shape[0] != pages):
        raise ValueError(f"{name}: the table's lengths must be [sequences] and refs [pages of the cache]")
    return rows.contiguous(), lengths.contiguous(), refs.contiguous()


def _each(t, sequences, device, name, what):
    """An int32 [sequences] argument, or None."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.shape != (sequences,):
        raise TypeError(f"{name}: {what} must be int32 [sequences]")
    if t.device != device:
        raise ValueError("all tensors must be on the same device")
    return t.contiguous()


_entries = {}


def _call(name, device, *args):
    """Run entry point ``name`` on ``device``'s current stream (appended as the last argument)."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(_lib.cache_lib(), name)
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _lib.check(status, name)


def _workspace(name, device, *sizes):
    """A workspace for ``name`` at these sizes: (tensor or None, bytes)."""
    need = getattr(_lib.cache_lib(), name + "_workspace")(*sizes)
    if need < 0:
        _lib.check(need, name)
    return (torch.empty(need, dtype=torch.uint8, device=device) if need else None), need


def _no_gradient(name, *tensors):
    if _differentiated(*(t for t in tensors if t is not None)):
        raise ValueError(f"{name} has no gradient: detach its inputs")


# ---------------------------------------------------------------- rows, attention
def cache_append(cache, table, k, v=None, *, counts=None):
    """Quantize rows k, v [sequences, tokens, kv_heads, head_dim] into the cache,
    in place: row j of a sequence at position lengths + j, for j < ``counts``
    (int32 [sequences]; default: all).  Codes and scales are
    ``quantize_cache_packed``'s, bit for bit.  Rows whose position has no page of
    the sequence's own (``cache_reserve``) are not written.  ``table.lengths``
    stays: the rows count as drafted until ``cache_accept``, or until the caller
    adds them to lengths.  ``v`` is None for a shared cache."""
    args, device = _cache_args(cache, "cache_append")
    _need_cuda(k, *(() if v is None else (v,)))
    dt = _float_type(k, "cache_append")
    if (v is None) != (cache.v_codes is None):
        raise ValueError("cache_append: v goes with a cache that has pools for the values")
    if k.dim() != 4 or k.shape[2:] != (args.kv_heads, args.head_dim) or k.device != device:
        raise ValueError("cache_append: k must be [sequences, tokens, kv_heads, head_dim], on the cache's device")
    if v is not None and (v.shape != k.shape or v.dtype != k.dtype):
        raise ValueError("cache_append: v must be like k")
    _no_gradient("cache_append", k, v)
    rows, lengths, refs = _table_args(table, args.pages, device, "cache_append")
    if k.shape[0] != rows.shape[0]:
        raise ValueError(f"cache_append: k has {k.shape[0]} sequences, the table {rows.shape[0]}")
    counts = _each(counts, rows.shape[0], device, "cache_append", "counts")
    k, v = k.contiguous(), None if v is None else v.contiguous()
    _call("cache_append", device, ctypes.byref(args), _ptr(rows), rows.shape[0], rows.shape[1], _ptr(lengths),
          _ptr(refs), _ptr(k), _ptr(v), dt, k.shape[1], _ptr(counts))


def cache_attention(q, cache, table, *, mask=None, counts=None, scale=None, return_lse=False):
    """Attention of new tokens over the cache: q [sequences, tokens, heads,
    head_dim] -> the same shape and type.  heads is a multiple of the cache's
    kv_heads.  The tokens' own rows are in the cache already, at positions
    lengths, lengths + 1, ... (``cache_append``).

    Token i attends to all cached positions and to the drafted tokens j with
    ``mask[i, j]`` (bool [tokens, tokens], or [sequences, tokens, tokens]: a tree
    of drafted tokens, each row true at the token itself and its ancestors), or
    with j <= i without a mask.  ``counts`` (int32 [sequences]): tokens from
    there on are padding.  ``scale``: default 1 / sqrt(head_dim); finite.

    Tokens with nothing to attend to get zeros.  Keys must be finite; a value past
    bf16's range is an infinity to the tokens that attend to it, a NaN is NaN, and
    neither reaches any other token.  With ``return_lse`` also the log
    of the softmax's sum, float32 [sequences, tokens, heads] (-inf there)."""
    args, device = _cache_args(cache, "cache_attention")
    _need_cuda(q)
    dt = _float_type(q, "cache_attention")
    if q.dim() != 4 or q.shape[3] != args.head_dim or q.device != device:
        raise ValueError("cache_attention: q must be [sequences, tokens, heads, head_dim], on the cache's device")
    B, T, H, D = q.shape
    if H == 0 or (args.kv_heads and H % args.kv_heads):        # (a cache without heads: the library's check)
        raise ValueError("cache_attention: heads must be a multiple of the cache's kv_heads")
    _no_gradient("cache_attention", q)
    rows, lengths, _ = _table_args(table, args.pages, device, "cache_attention")
    if rows.shape[0] != B:
        raise ValueError(f"cache_attention: q has {B} sequences, the table {rows.shape[0]}")
    counts = _each(counts, B, device, "cache_attention", "counts")
    if mask is not None:
        if mask.dtype != torch.bool or mask.shape not in ((T, T), (B, T, T)):
            raise TypeError("cache_attention: mask must be bool [tokens, tokens] or [sequences, tokens, tokens]")
        if mask.device != device:
            raise ValueError("all tensors must be on the same device")
        mask = mask.contiguous()
    q = q.contiguous()
    if q.data_ptr() & 15:
        q = q.clone()
    out = torch.empty_like(q)
    lse = torch.empty(B, T, H, dtype=torch.float32, device=device) if return_lse else None
    ref = ctypes.byref(args)
    work, need = _workspace("cache_attention", device, ref, B, rows.shape[1], dt, T, H)
    _call("cache_attention", device, ref, _ptr(rows), B, rows.shape[1], _ptr(lengths), _ptr(q), dt, T, H, _ptr(mask),
          int(mask is not None and mask.dim() == 3), _ptr(counts), 1 / math.sqrt(D) if scale is None else float(scale),
          _ptr(out), _ptr(lse), _ptr(work), need)
    return (out, lse) if return_lse else out


# -------------------------------------------------------------------- pages
def _fork(name, table, page_size, parents, children, keep, release):
    rows, lengths, refs = table
    device = rows.device
    out = PageTable(torch.empty((children, rows.shape[1]), dtype=torch.int32, device=device),
                    torch.empty(children, dtype=torch.int32, device=device), torch.empty_like(refs))
    _call("cache_fork", device, _ptr(rows), rows.shape[0], rows.shape[1], _ptr(lengths), _ptr(refs), refs.shape[0],
          page_size, _ptr(parents), children, _ptr(keep), int(release), *(_ptr(t) for t in out))
    return out


def cache_fork(table, parents, *, release=False):
    """The table of sequences that continue those of ``table``: sequence c of
    the result shares all pages of sequence ``parents[c]`` (int32 [children];
    one may have several children, or none).  The counts include both tables'
    entries, or with ``release`` only the new one's.  No row is copied:
    ``cache_reserve`` gives a sequence pages of its own in place of shared ones
    that it is about to write to, those reserved ahead among them."""
    _need_cuda(table.pages, parents)
    device = table.pages.device
    args = _table_args(table, None, device, "cache_fork")
    if parents.dtype != torch.int32 or parents.dim() != 1:
        raise TypeError("cache_fork: parents must be int32 [children]")
    # a page's size matters to the positions that are kept only, and all are
    return _fork("cache_fork", args, _PAGE_SIZES[0], parents.contiguous(), parents.shape[0], None, bool(release))


def cache_free(cache, table, keep=None):
    """The table after its sequences gave up their positions from ``keep`` on
    (int32 [sequences]; default: all of them), and the pages that held nothing
    else; pages that no sequence names any more are free."""
    args, device = _cache_args(cache, "cache_free")
    rows, lengths, refs = _table_args(table, args.pages, device, "cache_free")
    if keep is None:
        keep = torch.zeros_like(lengths)
    keep = _each(keep, rows.shape[0], device, "cache_free", "keep")
    return _fork("cache_free", (rows, lengths, refs), args.page_size, None, rows.shape[0], keep, True)


def cache_reserve(cache, table, tokens):
    """Pages of its own for the next ``tokens`` positions of every sequence (a
    number, or int32 [sequences]): free ones, in rising order, for entries that
    have none or one that other entries name too (its last holder keeps it).
    The cached rows of a partly filled last page come along.

    Returns (table, short): short int32 [sequences] is the number of pages a
    sequence still lacks (0: all there, and ``cache_append`` writes every row);
    ``cache_append`` leaves out the rows that they would hold."""
    args, device = _cache_args(cache, "cache_reserve")
    rows, lengths, refs = _table_args(table, args.pages, device, "cache_reserve")
    each = _each(tokens, rows.shape[0], device, "cache_reserve", "tokens") if isinstance(tokens, torch.Tensor) else None
    out, refs_out = torch.empty_like(rows), torch.empty_like(refs)
    short = torch.empty_like(lengths)
    work, need = _workspace("cache_reserve", device, rows.shape[0], rows.shape[1], args.pages)
    _call("cache_reserve", device, ctypes.byref(args), _ptr(rows), rows.shape[0], rows.shape[1], _ptr(lengths),
          _ptr(refs), 0 if each is not None else int(tokens), _ptr(each), _ptr(out), _ptr(refs_out), _ptr(short),
          _ptr(work), need)
    return PageTable(out, lengths, refs_out), short


def cache_accept(cache, table, accepted):
    """The drafted tokens that were accepted become cached ones: the rows of
    tokens ``accepted[b, 0], accepted[b, 1], ...`` (int32 [sequences, up to 64],
    rising, -1 behind the last) move together to positions lengths, lengths + 1,
    ..., in place, and the result's lengths include them.  A list ends before a
    token whose row or place has no page, or whose place is in a page that other
    sequences share (a table forked between the drafts and this call)."""
    args, device = _cache_args(cache, "cache_accept")
    rows, lengths, refs = _table_args(table, args.pages, device, "cache_accept")
    if accepted.dtype != torch.int32 or accepted.dim() != 2 or accepted.shape[0] != rows.shape[0]:
        raise TypeError("cache_accept: accepted must be int32 [sequences, up to 64]")
    if accepted.device != device:
        raise ValueError("all tensors must be on the same device")
    accepted = accepted.contiguous()
    out = torch.empty_like(lengths)
    _call("cache_accept", device, ctypes.byref(args), _ptr(rows), rows.shape[0], rows.shape[1], _ptr(lengths),
          _ptr(refs), _ptr(accepted), accepted.shape[1], _ptr(out))
    return PageTable(rows, out, refs)


def cache_compact(cache, table):
    """The pages in use moved to the front of the pools, in place: with n pages
    in use, those from n on go to the free ones below, both in rising order.
    ``table`` must hold every entry that names a page."""
    args, device = _cache_args(cache, "cache_compact")
    rows, lengths, refs = _table_args(table, args.pages, device, "cache_compact")
    out, refs_out = torch.empty_like(rows), torch.empty_like(refs)
    work, need = _workspace("cache_compact", device, args.pages)
    _call("cache_compact", device, ctypes.byref(args), _ptr(rows), rows.shape[0], rows.shape[1], _ptr(refs), _ptr(out),
          _ptr(refs_out), _ptr(work), need)
    return PageTable(out, lengths, refs_out)
