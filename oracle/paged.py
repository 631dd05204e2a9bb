"""A packed KV cache in pages, as include/mxq_pages.h defines it: NumPy, float64,
one sequence, one page and one row at a time.

Test infrastructure only (see ``oracle/__init__.py``).

A cache is a dict: fmt, block, and the pools k_codes, k_scales, v_codes,
v_scales (uint8 arrays; the v pools None where the values are the keys).  A
table is (pages, lengths, refs).  Operations return new tables and write the
pools in place.
"""

import numpy as np

from .cache import dequantize_cache_packed, quantize_cache_packed
from .formats import from_dtype_bits

POOLS = ("k_codes", "k_scales", "v_codes", "v_scales")


def _sizes(cache):
    pages, heads, size = cache["k_codes"].shape[:3]
    return pages, heads, size


def _values(codes, scales, cache):
    """float64 values of packed rows (exact: code values times powers of two or E4M3 scales fit float32)."""
    return from_dtype_bits(dequantize_cache_packed(codes, scales, cache["fmt"], cache["block"], "f32"), "f32")


def _cached(length, width, size):
    return min(max(int(length), 0), width * size)


def _place(cache, row, p):
    """(page, row within it) of position p, or None."""
    pages, _, size = _sizes(cache)
    slot = p // size
    if slot >= len(row) or not 0 <= row[slot] < pages:
        return None
    return int(row[slot]), p % size


def append(cache, table, k, v=None, counts=None):
    """k, v: float64 [B, T, heads, D]."""
    pages, lengths, refs = table
    for name, x in (("k", k), ("v", v)):
        if x is None:
            continue
        for b in range(x.shape[0]):
            n = _cached(lengths[b], pages.shape[1], _sizes(cache)[2])
            for j in range(x.shape[1] if counts is None else min(x.shape[1], int(counts[b]))):
                at = _place(cache, pages[b], n + j)
                if at is None or refs[at[0]] != 1:
                    continue
                codes, scales = quantize_cache_packed(x[b, j], cache["fmt"], cache["block"])
                cache[name + "_codes"][at[0], :, at[1]] = codes
                cache[name + "_scales"][at[0], :, at[1]] = scales


def attention(q, cache, table, mask=None, counts=None, scale=None):
    """q: float64 [B, T, H, D] -> out, lse, and per output what its rounding errors are bounded with: the largest
    sum |q_d k_d| over the positions a row attends to times scale, sum p |v| / sum p, the largest |v|, and how many
    positions."""
    pages, lengths, _ = table
    B, T, H, D = q.shape
    _, heads, size = _sizes(cache)
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, lse = np.zeros(q.shape), np.full((B, T, H), -np.inf)
    reach, mass, peak, met = np.zeros((B, T, H)), np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, T, H), int)
    for b in range(B):
        n = _cached(lengths[b], pages.shape[1], size)
        m = T if counts is None else min(max(int(counts[b]), 0), T)
        places = [_place(cache, pages[b], p) for p in range(n + m)]
        for i in range(m):
            see = [p for p in range(n + m) if places[p] is not None and (
                p < n or (p - n <= i if mask is None else bool((mask[b] if mask.ndim == 3 else mask)[i, p - n])))]
            if not see:
                continue
            pg, rw = np.array([places[p] for p in see]).T
            for g in range(heads):
                k = _values(cache["k_codes"][pg, g, rw], cache["k_scales"][pg, g, rw], cache)
                v = k if cache["v_codes"] is None else _values(cache["v_codes"][pg, g, rw], cache["v_scales"][pg, g, rw],
                                                               cache)
                for h in range(g * (H // heads), (g + 1) * (H // heads)):
                    s = scale * (k @ q[b, i, h])
                    e = np.exp(s - s.max())
                    out[b, i, h] = (e / e.sum()) @ v
                    lse[b, i, h] = s.max() + np.log(e.sum())
                    reach[b, i, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, i, h])).max()
                    mass[b, i, h] = (e / e.sum()) @ np.abs(v)
                    peak[b, i, h] = np.abs(v).max(0)
                    met[b, i, h] = len(see)
    return out, lse, reach, mass, peak, met


def _count(pages, n):
    flat = pages.reshape(-1)
    flat = flat[(flat >= 0) & (flat < n)]
    return np.bincount(flat, minlength=n).astype(np.int32)


def fork(table, parents, size, release=False, keep=None):
    pages, lengths, refs = table
    new = np.full((len(parents), pages.shape[1]), -1, np.int32)
    n = np.zeros(len(parents), np.int32)
    for c, parent in enumerate(parents):
        if not 0 <= parent < len(pages):
            continue
        n[c] = lengths[parent]
        row = [int(p) if 0 <= p < len(refs) else -1 for p in pages[parent]]
        if keep is not None:
            n[c] = min(n[c], max(int(keep[c]), 0))
            last = -(-max(int(n[c]), 0) // size)
            row = [p if i < last else -1 for i, p in enumerate(row)]
        new[c] = row
    return new, n, (refs + _count(new, len(refs)) - (_count(pages, len(refs)) if release else 0)).astype(np.int32)


def reserve(cache, table, tokens):
    """tokens: one number for each sequence."""
    pages, lengths, refs = table
    total, _, size = _sizes(cache)
    W = pages.shape[1]
    new = np.where((pages >= 0) & (pages < total), pages, -1).astype(np.int32)
    held, lack = refs.copy(), np.zeros(len(pages), np.int32)
    free = [p for p in range(total) if refs[p] <= 0]
    for b in range(len(pages)):
        n, t = _cached(lengths[b], W, size), max(int(tokens[b]), 0)
        end = -(-(n + t) // size)
        lack[b] = max(0, end - W)
        if t == 0:
            continue
        slot, filled = divmod(n, size)
        for i in range(slot, min(end, W)):
            old = new[b, i]
            if old >= 0 and held[old] <= 1:
                continue
            if not free:
                lack[b] += 1
                continue
            new[b, i] = free.pop(0)
            held[new[b, i]] = 1
            if old >= 0:                    # others name it too: what is cached of it comes along
                held[old] -= 1
                rows = filled if i == slot else 0
                for name in POOLS:
                    if cache[name] is not None:
                        cache[name][new[b, i], :, :rows] = cache[name][old, :, :rows]
    return (new, lengths.copy(), held), lack


def accept(cache, table, accepted):
    pages, lengths, refs = table
    size, W = _sizes(cache)[2], pages.shape[1]
    out = lengths.copy()
    for b in range(len(pages)):
        n, before, a = _cached(lengths[b], W, size), -1, 0
        for a in range(accepted.shape[1] + 1):
            if a == accepted.shape[1] or accepted[b, a] <= before:
                break
            src, dst = _place(cache, pages[b], n + int(accepted[b, a])), _place(cache, pages[b], n + a)
            if src is None or dst is None or refs[dst[0]] != 1:
                break
            for name in POOLS:
                if cache[name] is not None:
                    cache[name][dst[0], :, dst[1]] = cache[name][src[0], :, src[1]]
            before = accepted[b, a]
        out[b] = n + a
    return pages, out, refs


def compact(cache, table):
    pages, lengths, refs = table
    n = int((refs > 0).sum())
    free = [p for p in range(n) if refs[p] <= 0]
    to, held = {}, np.where(refs > 0, refs, 0).astype(np.int32)
    for p in range(n, len(refs)):
        if refs[p] > 0:
            to[p] = free.pop(0)
            held[to[p]], held[p] = refs[p], 0
            for name in POOLS:
                if cache[name] is not None:
                    cache[name][to[p]] = cache[name][p]
    move = [[(int(p) if p < n else to.get(int(p), -1)) if 0 <= p < len(refs) else -1 for p in row] for row in pages]
    return np.array(move, np.int32).reshape(pages.shape), lengths.copy(), held
