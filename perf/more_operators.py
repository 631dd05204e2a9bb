"""Cases of the paged packed cache: attention over it, rows written into it, and its pages.

Three operators, each timed as a user's program calls it:

* ``attend`` -- attention of new tokens (one of a decoding step, or a tree of drafted ones) over a cache whose keys and
  values are held as 8- or 4-bit codes in pages;
* ``append`` -- new rows quantized into their places in the pages;
* ``pages``  -- what a serving loop does to pages between two steps: ``fork`` (a beam step: sequences continue from their
  parents, shared last pages are copied before they are written), ``turnover`` (ended sequences free their pages, new ones
  get some), ``compact`` (a fragmented pool moved together) and ``accept`` (a verified path of a drafted tree moved
  together behind its context).

``run`` computes them in plain torch operations, or with the framework's kernels where ``own`` is true.  ``exact``
computes the same from the definitions, in 64 bits and sequence by sequence, written apart from the plain forms.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDPOINTS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# ------------------------------------------------------------------- cases
def _attend(name, seqs, tokens, heads, kv_heads, head_dim, fmt, block, context, page, tree, shared=False, dtype="bf16"):
    return dict(name=name, op="attend", seqs=seqs, tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim, fmt=fmt,
                block=block, context=context, page=page, tree=tree, shared=shared, dtype=dtype)


def _append(name, seqs, tokens, kv_heads, head_dim, fmt, block, context, page, shared=False, dtype="bf16"):
    return dict(name=name, op="append", seqs=seqs, tokens=tokens, kv_heads=kv_heads, head_dim=head_dim, fmt=fmt, block=block,
                context=context, page=page, shared=shared, dtype=dtype)


def _pages(name, kind, seqs, tokens, kv_heads, head_dim, fmt, block, context, page, group=1, shared=False):
    return dict(name=name, op="pages", kind=kind, seqs=seqs, tokens=tokens, kv_heads=kv_heads, head_dim=head_dim, fmt=fmt,
                block=block, context=context, page=page, group=group, shared=shared, dtype="bf16")


def listed():
    return [
        # one decoding step of four short conversations: latency
        _attend("attend_decode", 4, 1, 64, 8, 128, "fp8", 128, 2048, 64, False),
        # the same step of a full server: long contexts of very different lengths, keys and values in 4 bits
        _attend("attend_batch", 64, 1, 64, 8, 128, "mxfp4", 32, 16384, 128, False),
        # verification of a tree of sixteen drafted tokens, small pages
        _attend("attend_tree", 32, 16, 32, 8, 128, "nvfp4", 16, 8192, 16, True),
        # verification of large trees over long contexts: the products count
        _attend("attend_wide_tree", 8, 64, 64, 8, 128, "fp8", 32, 16384, 64, True),
        # one step over the [4, 8192, 512] cache of compressed keys, which are the values too
        _attend("attend_compressed", 4, 1, 64, 1, 512, "nvfp4", 16, 8192, 64, False, shared=True, dtype="f16"),
        # one decoding step's rows of 64 sequences
        _append("append_step", 64, 1, 8, 128, "fp8", 128, 2048, 64),
        # prompts of four sequences, of different lengths
        _append("append_prompt", 4, 8192, 8, 128, "mxfp4", 32, 8192, 128),
        # a step of beam search, four beams each
        _pages("fork_step", "fork", 64, 1, 8, 128, "fp8", 128, 1024, 64, group=4),
        # the same with many long beams over compressed keys
        _pages("fork_long", "fork", 256, 4, 1, 512, "nvfp4", 16, 16384, 256, group=8, shared=True),
        # a serving step at which an eighth of the sequences ended and others began
        _pages("turnover", "turnover", 128, 16, 8, 128, "mxfp4", 32, 2048, 16),
        # a fragmented pool moved together
        _pages("compact", "compact", 64, 1, 8, 128, "fp8", 32, 1024, 32),
        # drafted rows written, and the accepted ones moved together
        _pages("accept", "accept", 32, 16, 8, 128, "fp8", 128, 1024, 64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "pages"])
    fmt, block = rng.choice([("fp8", 16), ("fp8", 32), ("fp8", 64), ("fp8", 128), ("mxfp4", 32), ("mxfp4", 64), ("nvfp4", 16), ("nvfp4", 16)])
    head_dim = rng.choice([64, 128, 128, 256, 512])
    block = min(block, head_dim)
    page = rng.choice([16, 32, 64, 128, 256])
    shared, dtype = rng.random() < 0.25, rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "attend":
        kv_heads, group = rng.choice([(8, 1), (1, 12), (2, 8), (8, 4), (8, 8), (4, 7), (1, 64), (8, 5), (1, 16)])
        seqs, tokens = _log_int(rng, 1, 64), 1 if rng.random() < 0.4 else _log_int(rng, 2, 64)
        # no more than the largest listed case reads or multiplies
        most = min((1 << 28) // (seqs * kv_heads * head_dim), (1 << 35) // (seqs * kv_heads * group * tokens * head_dim), 32768)
        return dict(op=op, seqs=seqs, tokens=tokens, heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, fmt=fmt, block=block,
                    context=_log_int(rng, 1, max(1, most)), page=page, tree=tokens > 1 and rng.random() < 0.7, shared=shared, dtype=dtype)
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "append":
        seqs, tokens = _log_int(rng, 1, 64), _log_int(rng, 1, 4096)
        tokens = max(1, min(tokens, (1 << 23) // (seqs * kv_heads * head_dim)))
        return dict(op=op, seqs=seqs, tokens=tokens, kv_heads=kv_heads, head_dim=head_dim, fmt=fmt, block=block,
                    context=max(tokens, _log_int(rng, 1, 1024)), page=page, shared=shared, dtype=dtype)
    kind, group, seqs = rng.choice(["fork", "turnover", "compact", "accept"]), rng.choice([1, 2, 4, 8]), _log_int(rng, 1, 128)
    most = max(1, (1 << 25) // (seqs * kv_heads * head_dim))
    return dict(op=op, kind=kind, seqs=seqs * (group if kind == "fork" and seqs * group <= 256 else 1), tokens=_log_int(rng, 1, 32), kv_heads=kv_heads, head_dim=head_dim,
                fmt=fmt, block=block, context=_log_int(rng, 1, min(4096, most)), page=page,
                group=group if kind == "fork" and seqs * group <= 256 else 1, shared=shared, dtype=dtype)


# ------------------------------------------------------------- plain codec
def _quantize(x, fmt, block):
    """Codes and scale bytes of groups of channels: a power-of-two scale no smaller than amax / the format's largest value."""
    b = x.float().unflatten(-1, (-1, block))
    ratio = (b.abs().amax(-1, keepdim=True) / (448.0 if fmt == "fp8" else 6.0)).clamp_min(2.0 ** -126)
    mant, expo = torch.frexp(ratio)
    expo = expo - (mant == 0.5).to(expo.dtype)
    if fmt == "nvfp4":
        expo = expo.clamp(-9, 8)
    scale = torch.exp2(expo.float())
    v = b / scale
    scales = scale.squeeze(-1).to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "nvfp4" else (expo.squeeze(-1) + 127).to(torch.uint8)
    if fmt == "fp8":
        return v.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8), scales
    # nearest value, a tie to the code that is even: a midpoint counts for the code above it where that one is even
    mag, code = v.abs(), torch.zeros_like(v, dtype=torch.uint8)
    for k, mid in enumerate(MIDPOINTS):
        code += (mag >= mid if k % 2 else mag > mid).to(torch.uint8)
    code = (code | (v < 0).to(torch.uint8) << 3).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, scales


def _dequantize(codes, scales, fmt):
    """float32 values of codes [..., D or D / 2] with scales [..., D / block]."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
        v = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.exp2(scales.float() - 127)
    return (v.unflatten(-1, (s.shape[-1], -1)) * s[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _randint(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _rows(g, case, *lead):
    """Keys or values [..., kv_heads, D] of normal numbers: some channels are larger than others."""
    liked = torch.exp2(_randint(g, -1, 3, case["kv_heads"], case["head_dim"]).float() / 2)
    return _randn(g, *lead, case["kv_heads"], case["head_dim"]) * liked


def _pool(g, case, pages):
    """Codes and scales of `pages` pages, quantized a part at a time."""
    made = [_quantize(_rows(g, case, n, case["page"]).transpose(1, 2), case["fmt"], case["block"])
            for n in _parts(pages, max(1, (1 << 26) // (case["kv_heads"] * case["page"] * case["head_dim"])))]
    return torch.cat([c for c, _ in made]), torch.cat([s for _, s in made])


def _parts(n, most):
    return [min(most, n - at) for at in range(0, n, most)]


def _ancestors(g, seqs, tokens):
    """mask[b, i, j]: whether drafted token j is i itself or one of those before it in a random tree."""
    i = torch.arange(tokens, device="cuda")
    parent = (torch.rand(seqs, tokens, generator=g, device="cuda") * i).long()
    reach = torch.eye(tokens, device="cuda").repeat(seqs, 1, 1)
    reach.scatter_(2, parent[..., None], 1.0)
    while tokens > 1:
        further = ((reach @ reach) > 0).float()
        if torch.equal(further, reach):
            break
        reach = further
    return reach > 0


def _lengths(g, case):
    """Contexts of different lengths, the longest of them the case's."""
    n = (torch.rand(case["seqs"], generator=g, device="cuda") * 0.9 + 0.1) * case["context"]
    n[0] = case["context"]
    return n.to(torch.int32)


def _table(g, case, need, spare):
    """Pages of sequences that need `need` positions each, anywhere in a pool that holds as many of the longest and `spare` more."""
    P, B = case["page"], case["seqs"]
    width = -(-(case["context"] + case["tokens"]) // P)
    slots = torch.arange(width, device="cuda") < ((need + P - 1) // P)[:, None]
    own_pages = torch.cumsum(slots.reshape(-1), 0).view(B, width) - 1
    order = torch.randperm(B * width + spare, generator=g, device="cuda").to(torch.int32)
    table = torch.where(slots, order[own_pages.clamp_min(0)], -1).contiguous()
    return table, _counts(table, B * width + spare)


def _counts(table, pages):
    flat = table.reshape(-1).long()
    return torch.bincount(torch.where(flat < 0, pages, flat), minlength=pages + 1)[:pages].to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s, dt = dict(case=case), DTYPES[case["dtype"]]
    B, T, D = case["seqs"], case["tokens"], case["head_dim"]
    s["lengths"] = _lengths(g, case)
    s["counts"] = None
    if case["op"] == "append":
        s["lengths"] = s["lengths"] - s["lengths"].clamp_max(T)          # prompts start where nothing, or a part, is cached
        if T > 1:
            s["counts"] = torch.minimum(_lengths(g, dict(case, context=T)), torch.tensor(T, device="cuda", dtype=torch.int32))
    if case["op"] == "attend" and T > 1 and B > 1:
        s["counts"] = T - _randint(g, 0, 2, B) * _randint(g, 0, max(1, T // 2), B)
    need = s["lengths"] + (T if case["op"] != "pages" or case["kind"] == "accept" else 0)
    s["table"], s["refs"] = _table(g, case, need, 2 * B if case.get("kind") == "fork" else 8)
    if case["op"] == "pages":
        _prepare_pages(g, s)
    for name in ("k", "v"):
        pair = (None, None) if name == "v" and case["shared"] else _pool(g, case, s["refs"].numel())
        s[name + "_codes"], s[name + "_scales"] = pair
    if case["op"] == "append" or case.get("kind") == "accept":
        s["k"] = _rows(g, case, B, T).to(dt)
        s["v"] = None if case["shared"] else _rows(g, case, B, T).to(dt)
    if case["op"] == "attend":
        s["q"] = (_randn(g, B, T, case["heads"], D) * 0.7).to(dt)
        s["mask"] = _ancestors(g, B, T) if case["tree"] else None
    return s


def _prepare_pages(g, s):
    c = s["case"]
    B, T = c["seqs"], c["tokens"]
    if c["kind"] == "fork":
        # beams of a group share the pages of the first three quarters, and each continues from a beam of its group
        first = torch.arange(B, device="cuda") // c["group"] * c["group"]
        s["lengths"] = s["lengths"][first].contiguous()
        common = torch.arange(s["table"].shape[1], device="cuda") < (s["lengths"] * 3 // 4 // c["page"])[:, None]
        grown = s["table"][first]                              # the first beam's pages: as many as the others need
        s["table"] = torch.where(common | (s["table"] < 0) & (grown >= 0), grown, s["table"])
        s["table"] = torch.where(grown < 0, -1, s["table"]).contiguous()
        s["refs"] = _counts(s["table"], s["refs"].numel())
        s["parents"] = (first + (torch.rand(B, generator=g, device="cuda") * torch.clamp(B - first, max=c["group"])).long()).to(torch.int32)
    elif c["kind"] == "turnover":
        ended = torch.rand(B, generator=g, device="cuda") < 0.125
        s["keep"] = torch.where(ended, 0, s["lengths"])
        s["new"] = torch.where(ended, _lengths(g, c), T).to(torch.int32)
    elif c["kind"] == "compact":
        # half of the sequences ended
        s["table"] = torch.where((torch.rand(B, generator=g, device="cuda") < 0.5)[:, None], s["table"], -1).contiguous()
        s["lengths"] = torch.where((s["table"] >= 0).any(1), s["lengths"], 0)
        s["refs"] = _counts(s["table"], s["refs"].numel())
    else:
        # a path through the tree: rising draft numbers, -1 behind the last
        reach = _ancestors(g, B, T)
        leaf = _randint(g, 0, T, B).long()
        path = reach[torch.arange(B, device="cuda"), leaf]
        order = torch.where(path, torch.arange(T, device="cuda"), T).sort(1).values
        s["accepted"] = torch.where(order < T, order, -1)[:, : min(T, 12)].to(torch.int32).contiguous()


# ------------------------------------------------------------- plain forms
def _pools(s):
    """The pools as outputs: fp8 codes and all scales as the values they stand for, pairs of 4-bit codes as they are stored."""
    fmt = s["case"]["fmt"]
    out = []
    for name in ("k", "v"):
        if s[name + "_codes"] is not None:
            codes, scales = s[name + "_codes"], s[name + "_scales"]
            out += [codes.view(torch.float8_e4m3fn) if fmt == "fp8" else codes,
                    scales.view(torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu)]
    return out


def _gathered(s, name):
    """float32 rows [B, kv_heads, positions, D] of every sequence's pages."""
    codes, scales = s[name + "_codes"], s[name + "_scales"]
    at = s["table"].clamp_min(0).long()
    rows = _dequantize(codes[at], scales[at], s["case"]["fmt"])
    return rows.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c, q = s["case"], s["q"]
    B, T, H, D = q.shape
    Hk, G = c["kv_heads"], H // c["kv_heads"]
    k = _gathered(s, "k")
    v = k if s["v_codes"] is None else _gathered(s, "v")
    pos, n = torch.arange(k.shape[2], device="cuda"), s["lengths"][:, None]
    count = T if s["counts"] is None else s["counts"][:, None]
    known, drafted = pos < n, (pos >= n) & (pos < n + count)
    tree = torch.ones(T, T, dtype=torch.bool, device="cuda").tril().expand(B, T, T) if s["mask"] is None else s["mask"]
    may = tree.gather(2, (pos - n).clamp(0, T - 1).long()[:, None, :].expand(B, T, -1)) & drafted[:, None, :]
    may = (may | known[:, None, :]) & (s["table"] >= 0).repeat_interleave(c["page"], 1)[:, None, :]
    if s["counts"] is not None:
        may = may & (torch.arange(T, device="cuda") < count)[..., None]
    may = may[:, None, :, None, :].expand(B, 1, T, G, -1).flatten(2, 3)
    rows = q.float().view(B, T, Hk, G, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.where(may, rows @ k.transpose(2, 3) * (1 / math.sqrt(D)), -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(3, keepdim=True)
    out = torch.where(total > 0, p @ v / total, 0.0)
    lse = (top + torch.log(total)).squeeze(3)
    out = out.view(B, Hk, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D).to(q.dtype)
    return [out, lse.view(B, Hk, T, G).permute(0, 2, 1, 3).reshape(B, T, H)]


def _plain_append(s):
    c = s["case"]
    B, T, P = c["seqs"], c["tokens"], c["page"]
    j = torch.arange(T, device="cuda")
    pos = s["lengths"][:, None] + j
    slot = pos // P
    fits = slot < s["table"].shape[1]
    page = s["table"].gather(1, torch.where(fits, slot, 0).long()).long()
    real = fits & (page >= 0)
    if s["counts"] is not None:
        real = real & (j < s["counts"][:, None])
    page, row = page[real], (pos % P)[real].long()
    for name in ("k", "v"):
        if s[name] is not None:
            codes, scales = _quantize(s[name][real], c["fmt"], c["block"])
            s[name + "_codes"][page, :, row] = codes
            s[name + "_scales"][page, :, row] = scales
    return _pools(s)


def _plain_fork(table, lengths, refs, parents, keep, P):
    """Rows of the table from their parents, cut to `keep` positions; refs follow, the old rows given up."""
    new, n = table[parents.long()], lengths[parents.long()]
    if keep is not None:
        n = torch.minimum(n, keep)
        new = torch.where(torch.arange(new.shape[1], device="cuda") < ((n + P - 1) // P)[:, None], new, -1)
    return new, n, refs + _counts(new, refs.numel()) - _counts(table, refs.numel())


def _plain_reserve(s, table, lengths, refs, tokens):
    c = s["case"]
    B, W, P = table.shape[0], table.shape[1], c["page"]
    slot = torch.arange(W, device="cuda")
    need = (lengths + tokens + P - 1) // P
    missing = (table < 0) & (slot < need[:, None])
    # the page that the next row goes to: copied where others hold it too, all but the last of those that ask
    at = (lengths // P).clamp_max(W - 1).long()[:, None]
    last = table.gather(1, at).squeeze(1)
    ask = (lengths % P > 0) & (lengths // P < W) & (last >= 0)
    ask = ask & (torch.as_tensor(tokens, device="cuda") > 0)
    same = (last[:, None] == last[None, :]) & ask[:, None] & ask[None, :]
    before = same.tril(-1).sum(1)
    copy = ask & (before < refs[last.clamp_min(0).long()] - 1)
    want = torch.cat([copy[:, None], missing], 1)
    rank = torch.cumsum(want.reshape(-1), 0).view(B, W + 1) - 1
    order = torch.argsort((refs > 0).int(), stable=True)
    got = want & (rank < (refs <= 0).sum())
    page = torch.where(got, order[rank.clamp(0, order.numel() - 1)], -1).to(torch.int32)
    new = torch.where(got[:, 1:], page[:, 1:], table)
    new = torch.where((slot == at) & got[:, :1], page[:, :1], new)
    refs = refs - _counts(torch.where(got[:, 0], last, -1), refs.numel()) + _counts(page, refs.numel())
    moved = got[:, 0]
    src, dst = last[moved].long(), page[:, 0][moved].long()
    below = (torch.arange(P, device="cuda") < (lengths % P)[moved][:, None])[:, None, :, None]
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        if s[name] is not None:
            s[name][dst] = torch.where(below, s[name][src], s[name][dst])
    # what could not be had: pages, room in the table, and the last holder's page where a copy of another's failed
    short = want.sum(1) - got.sum(1) + (need - W).clamp_min(0) + (ask & ~copy & (refs[last.clamp_min(0).long()] > 1))
    return new, refs, short.to(torch.int32)


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    N = refs.numel()
    used = refs > 0
    n = used.sum()
    i = torch.arange(N, device="cuda")
    src, dst = i[used & (i >= n)], i[~used & (i < n)]
    to = i.to(torch.int32)
    to[src] = dst.to(torch.int32)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        if s[name] is not None:
            s[name][dst] = s[name][src]
    new = refs.clone()
    new[dst], new[src] = refs[src], 0
    return [torch.where(table >= 0, to[table.clamp_min(0).long()], -1), s["lengths"], new, *_pools(s)]


def _plain_accept(s):
    c = s["case"]
    _plain_append(s)
    A, P = s["accepted"].shape[1], c["page"]
    good = s["accepted"] >= 0
    a = torch.arange(A, device="cuda").expand_as(good)
    src, dst = (s["lengths"][:, None] + s["accepted"])[good], (s["lengths"][:, None] + a)[good]
    b = torch.arange(c["seqs"], device="cuda")[:, None].expand_as(good)[good]
    src_page, dst_page = s["table"][b, (src // P).long()].long(), s["table"][b, (dst // P).long()].long()
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        if s[name] is not None:
            s[name][dst_page, :, (dst % P).long()] = s[name][src_page, :, (src % P).long()]
    return [s["table"], s["lengths"] + good.sum(1, dtype=torch.int32), s["refs"], *_pools(s)]


def _plain_pages(s):
    c = s["case"]
    table, lengths, refs = s["table"], s["lengths"], s["refs"]
    if c["kind"] == "compact":
        return _plain_compact(s)
    if c["kind"] == "accept":
        return _plain_accept(s)
    if c["kind"] == "fork":
        table, lengths, refs = _plain_fork(table, lengths, refs, s["parents"], None, c["page"])
        tokens = c["tokens"]
    else:
        table, lengths, refs = _plain_fork(table, lengths, refs, torch.arange(c["seqs"], device="cuda"), s["keep"], c["page"])
        tokens = s["new"]
    table, refs, short = _plain_reserve(s, table, lengths, refs, tokens)
    return [table, lengths, refs, short, *_pools(s)]


_PLAIN = {"attend": _plain_attend, "append": _plain_append, "pages": _plain_pages}


# ---------------------------------------------------------- framework's calls
def _own_attend(mxq, s, cache, table):
    return list(mxq.cache_attention(s["q"], cache, table, mask=s["mask"], counts=s["counts"], return_lse=True))


def _own_append(mxq, s, cache, table):
    mxq.cache_append(cache, table, s["k"], s["v"], counts=s["counts"])
    return _pools(s)


def _own_pages(mxq, s, cache, table):
    kind = s["case"]["kind"]
    if kind == "compact":
        return [*mxq.cache_compact(cache, table), *_pools(s)]
    if kind == "accept":
        mxq.cache_append(cache, table, s["k"], s["v"])
        return [*mxq.cache_accept(cache, table, s["accepted"]), *_pools(s)]
    if kind == "fork":
        table, short = mxq.cache_reserve(cache, mxq.cache_fork(table, s["parents"], release=True), s["case"]["tokens"])
    else:
        table, short = mxq.cache_reserve(cache, mxq.cache_free(cache, table, keep=s["keep"]), s["new"])
    return [*table, short, *_pools(s)]


_OWN = {"attend": _own_attend, "append": _own_append, "pages": _own_pages}


def run(state):
    op = state["case"]["op"]
    if own:
        import nvfp4_quantization_grouped_amd as mxq
        cache = mxq.PagedCache(state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"], state["case"]["fmt"])
        return _OWN[op](mxq, state, cache, mxq.PageTable(state["table"], state["lengths"], state["refs"]))
    return _PLAIN[op](state)


# --------------------------------------------------------------------- work
def work(case):
    B, T, Hk, D, P = (case[n] for n in ("seqs", "tokens", "kv_heads", "head_dim", "page"))
    b = BYTES[case["dtype"]]
    row = D * (1.0 if case["fmt"] == "fp8" else 0.5) + D / case["block"]         # a key's or value's codes and scales
    kinds = 1 if case["shared"] else 2
    cached = case["context"] * (1 + 0.55 * (B - 1))                       # positions of all sequences, on average
    width = -(-(case["context"] + T) // P)
    if case["op"] == "attend":
        H = case["heads"]
        rows = B * T * H
        return {"bytes": cached * Hk * kinds * row + rows * (2 * D * b + 4) + B * width * 4, "flops": 4 * cached * T * H * D}
    if case["op"] == "append":
        n = B * T * (0.55 if T > 1 else 1) * Hk * kinds
        return {"bytes": n * (D * b + row), "flops": 4 * n * D}
    tables = 2 * B * width * 4 + 8 * (cached / P + B)
    if case["kind"] == "accept":
        n = B * T * Hk * kinds
        return {"bytes": n * (D * b + row) + 2 * B * min(T, 3) * Hk * kinds * row + tables, "flops": 4 * n * D}
    moved = {"fork": 0.6 * B * P / 2, "turnover": 0, "compact": 0.36 * cached}[case["kind"]]    # rows that change their page
    return {"bytes": 2 * moved * Hk * kinds * row + tables, "flops": B * width}


# ------------------------------------------------------- definitions, 64 bits
def _decoded(codes, scales, fmt):
    """float64 values, from the bits of each code: sign, exponent, mantissa."""
    if fmt != "fp8":
        codes = torch.stack([codes % 16, codes // 16], -1).flatten(-2)
    c = codes.to(torch.int64)
    bits, bias = (3, 7) if fmt == "fp8" else (1, 1)
    sign = 1.0 - 2.0 * ((c >> (7 if fmt == "fp8" else 3)) & 1).double()
    expo, mant = (c >> bits) & (15 if fmt == "fp8" else 3), (c & (2 ** bits - 1)).double() / 2 ** bits
    v = sign * torch.where(expo > 0, (1 + mant) * torch.exp2((expo - bias).double()), mant * 2.0 ** (1 - bias))
    z = scales.to(torch.int64)
    if fmt == "nvfp4":
        e, m = z >> 3, (z & 7).double() / 8
        s = torch.where(e > 0, (1 + m) * torch.exp2((e - 7).double()), m * 2.0 ** -6)
    else:
        s = torch.exp2((z - 127).double())
    return v * s.repeat_interleave(v.shape[-1] // s.shape[-1], -1)


def _exact_attend(s):
    c, q = s["case"], s["q"].to(torch.float64)
    B, T, H, D = q.shape
    G, P = H // c["kv_heads"], c["page"]
    out = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    lengths = s["lengths"].tolist()
    counts = [T] * B if s["counts"] is None else s["counts"].tolist()
    for b in range(B):
        n, m = lengths[b], counts[b]
        pages = s["table"][b, : -(-(n + m) // P)].long()
        k = _decoded(s["k_codes"][pages], s["k_scales"][pages], c["fmt"]).transpose(0, 1).flatten(1, 2)[:, : n + m]
        v = k if c["shared"] else _decoded(s["v_codes"][pages], s["v_scales"][pages], c["fmt"]).transpose(0, 1).flatten(1, 2)[:, : n + m]
        hidden = ~s["mask"][b, :m, :m] if s["mask"] is not None else torch.ones(m, m, device="cuda", dtype=torch.bool).triu(1)
        hidden = torch.cat([hidden.new_zeros(m, n), hidden], 1)
        for h in range(c["kv_heads"]):
            x = torch.einsum("ihd,pd->ihp", q[b, :m, h * G:(h + 1) * G], k[h]) / math.sqrt(D)
            x.masked_fill_(hidden[:, None, :], -math.inf)
            lse[b, :m, h * G:(h + 1) * G] = torch.logsumexp(x, 2)
            out[b, :m, h * G:(h + 1) * G] = torch.einsum("ihp,pd->ihd", torch.softmax(x, 2).nan_to_num(0.0), v[h])
    return [out, lse]


def _exact_codes(x, fmt, block):
    """Codes (as values for fp8, as stored for the 4-bit formats) and scales as values."""
    v = x.to(torch.float64).unflatten(-1, (-1, block))
    most = 448.0 if fmt == "fp8" else 6.0
    low, high = (-9, 8) if fmt == "nvfp4" else (-126, 127)
    top = v.abs().max(-1, keepdim=True).values
    power = torch.ceil(torch.log2(top.clamp_min(2.0 ** -160) / most)).clamp(low, high)
    power = torch.where(torch.exp2(power - 1) * most >= top, (power - 1).clamp_min(low), power)
    power = torch.where(torch.exp2(power) * most < top, (power + 1).clamp_max(high), power)
    scale = torch.exp2(power)
    u = v / scale
    mag = u.abs().clamp_max(most)
    unit = 2.0 ** -6 if fmt == "fp8" else 1.0                           # the smallest normal value; below it the step stays
    e = torch.floor(torch.log2(mag.clamp_min(unit)))
    e = torch.where(torch.exp2(e) > mag.clamp_min(unit), e - 1, e)
    step = torch.exp2(e - (3 if fmt == "fp8" else 1))
    r = torch.round(mag / step) * step
    if fmt == "fp8":
        return (torch.copysign(r, u)).flatten(-2), scale.squeeze(-1)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    code = (torch.searchsorted(grid, r.contiguous()) + 8 * (u < 0)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.squeeze(-1)


def _exact_pools(s):
    """The pools as floats where _pools returns values, copies that the definitions below write to."""
    fmt, out = s["case"]["fmt"], []
    for codes, scales in ((s["k_codes"], s["k_scales"]), (s["v_codes"], s["v_scales"])):
        if codes is not None:
            out += [codes.view(torch.float8_e4m3fn).float() if fmt == "fp8" else codes.clone(),
                    scales.view(torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu).float()]
    return out


def _exact_append(s, pools=None):
    c = s["case"]
    pools = _exact_pools(s) if pools is None else pools
    table, lengths = s["table"].tolist(), s["lengths"].tolist()
    counts = [c["tokens"]] * c["seqs"] if s["counts"] is None else s["counts"].tolist()
    for which, x in enumerate((s["k"], s["v"])):
        if x is None:
            continue
        for b in range(c["seqs"]):
            codes, scales = _exact_codes(x[b], c["fmt"], c["block"])
            at = 0
            while at < counts[b]:                   # the part of a page that the rows fill
                slot, row = divmod(lengths[b] + at, c["page"])
                n = min(c["page"] - row, counts[b] - at)
                page = table[b][slot]
                pools[2 * which][page, :, row:row + n] = codes[at:at + n].transpose(0, 1).to(pools[2 * which].dtype)
                pools[2 * which + 1][page, :, row:row + n] = scales[at:at + n].transpose(0, 1).float()
                at += n
    return pools


def _exact_pages(s):
    """Sequence by sequence, page by page."""
    c = s["case"]
    P, B = c["page"], c["seqs"]
    table, lengths, refs = s["table"].tolist(), s["lengths"].tolist(), s["refs"].tolist()
    pools = _exact_append(s) if c["kind"] == "accept" else _exact_pools(s)
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if c["kind"] == "accept":
        for b, path in enumerate(s["accepted"].tolist()):
            path = [a for a in path if a >= 0]
            for n, a in enumerate(path):
                (i, x), (j, y) = divmod(lengths[b] + a, P), divmod(lengths[b] + n, P)
                for pool in pools:
                    pool[table[b][j], :, y] = pool[table[b][i], :, x]
            lengths[b] += len(path)
        return [whole(table), whole(lengths), whole(refs), *pools]
    if c["kind"] == "compact":
        n, low, to = sum(r > 0 for r in refs), 0, {}
        for page in range(n, len(refs)):
            if refs[page] > 0:
                while refs[low] > 0:
                    low += 1
                to[page], refs[low], refs[page] = low, refs[page], 0
                for pool in pools:
                    pool[low] = pool[page]
        table = [[to.get(p, p) for p in row] for row in table]
        return [whole(table), whole(lengths), whole(refs), *pools]
    if c["kind"] == "fork":
        parents, keep, tokens = s["parents"].tolist(), None, [c["tokens"]] * B
    else:
        parents, keep, tokens = list(range(B)), s["keep"].tolist(), s["new"].tolist()
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] -= 1
    table, lengths = [list(table[p]) for p in parents], [lengths[p] for p in parents]
    for b, row in enumerate(table):
        if keep is not None:
            lengths[b] = min(lengths[b], keep[b])
            for i in range(-(-lengths[b] // P), len(row)):
                row[i] = -1
        for p in row:
            if p >= 0:
                refs[p] += 1
    free = [p for p, r in enumerate(refs) if r == 0]
    short = [0] * B
    for b, row in enumerate(table):
        short[b] = max(0, -(-(lengths[b] + tokens[b]) // P) - len(row))
        slot, filled = divmod(lengths[b], P)
        if filled and tokens[b] > 0 and slot < len(row) and row[slot] >= 0 and refs[row[slot]] > 1:
            if free:
                page = free.pop(0)
                for pool in pools:
                    pool[page, :, :filled] = pool[row[slot], :, :filled]
                refs[row[slot]] -= 1
                row[slot], refs[page] = page, 1
            else:
                short[b] += 1
        for i in range(min(len(row), -(-(lengths[b] + tokens[b]) // P))):
            if row[i] < 0 and free:
                row[i] = free.pop(0)
                refs[row[i]] = 1
            elif row[i] < 0:
                short[b] += 1
    return [whole(table), whole(lengths), whole(refs), whole(short), *pools]


_EXACT = {"attend": _exact_attend, "append": _exact_append, "pages": _exact_pages}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
