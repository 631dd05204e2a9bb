"""cache_reserve where pages were reserved ahead and are shared, against the
oracle and against rows that are kept apart from any table: what lacks nothing
can be written, and is what attention reads."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
import oracle
from oracle import paged
from tests.gpu_util import dev
from tests.moe_util import f64
from tests.paged_util import (assert_same_pools, assert_same_table, check_attention, copied, counted, on_gpu, pools,
                              table_of, table_on_gpu, values)

pytestmark = pytest.mark.gpu

i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev())  # noqa: E731


def table_ahead(g, B, W, size, pages, most):
    """Sequences with pages up to `most` slots past their rows, many of them shared with the one before or with the first."""
    lengths = g.integers(0, W * size + 1, B)
    lengths[g.random(B) < 0.3] //= size
    lengths[g.random(B) < 0.5] //= size
    lengths[g.random(B) < 0.3] *= size
    lengths = np.minimum(lengths, W * size)
    rows = np.full((B, W), -1, np.int32)
    order = list(g.permutation(pages))
    for b in range(B):
        for i in range(min(W, -(-lengths[b] // size) + g.integers(0, most + 1))):
            from_ = rows[0 if g.random() < 0.3 else b - 1, i] if b and g.random() < 0.7 else -1
            if from_ >= 0:
                rows[b, i] = from_
            elif order and g.random() < 0.9:
                rows[b, i] = order.pop()
    return counted(rows, lengths, pages)


def held_alone(got, lack, lengths, tokens, size):
    pages, refs = got.pages.cpu().numpy(), got.refs.cpu().numpy()
    for b, n in enumerate(np.maximum(lengths, 0)):
        if tokens[b] > 0 and lack[b] == 0:
            entries = pages[b, n // size: -(-(int(n) + int(tokens[b])) // size)]
            assert (entries >= 0).all() and (refs[entries] == 1).all(), (b, entries)


def check(cache, table, tokens, what):
    gpu = on_gpu(cache)
    got, lack = mxq.cache_reserve(gpu, table_on_gpu(table), i32(tokens))
    want, want_lack = paged.reserve(cache, table, tokens)
    assert_same_table(got, want, what)
    assert lack.tolist() == want_lack.tolist(), what
    assert_same_pools(gpu, cache, what)
    held_alone(got, want_lack, table[1], tokens, cache["k_codes"].shape[2])


@pytest.mark.parametrize("B,W,size,pages,most", [
    (1, 3, 16, 9, 2), (2, 4, 16, 30, 3), (3, 9, 32, 60, 8), (17, 5, 64, 150, 3), (65, 70, 16, 3000, 60), (70, 12, 16, 900, 5),
    (1030, 4, 16, 4000, 3), (2100, 3, 16, 3000, 2)])
@pytest.mark.parametrize("seed", range(3))
def test_shared_pages_ahead(B, W, size, pages, most, seed):
    g = np.random.default_rng(seed * 100 + B)
    few = pages > 400
    cache = pools(g, pages, 1 if few else 3, size, 64, "nvfp4" if few else "fp8", 16 if few else 64, few)
    table = table_ahead(g, B, W, size, pages, most)
    tokens = g.integers(-1, most * size + 2, B) * (g.random(B) < 0.8)
    check(cache, table, tokens, "ahead")


@pytest.mark.parametrize("free", [0, 1, 2, 5, 11, 40])
@pytest.mark.parametrize("B", [3, 9, 130])
def test_the_pool_runs_out(B, free):
    g = np.random.default_rng(free + B)
    cache = pools(g, 200, 1, 16, 64, "fp8", 32)
    table = table_ahead(g, B, 6, 16, 200, 4)
    refs = table[2].copy()
    refs[np.flatnonzero(refs == 0)[free:]] = 1           # held by somebody else
    check(cache, (table[0], table[1], refs), g.integers(0, 60, B), "short of pages")


def test_the_same_page_twice_and_pages_of_others():
    g = np.random.default_rng(0)
    cache = pools(g, 12, 2, 32, 128, "mxfp4", 32)
    rows = np.array([[0, 3, 3, 3], [3, 5, -1, 5], [1 << 30, 5, 7, -9]], np.int32)
    table = counted(rows, [32, 40, 20], 12)
    table[2][7] = 2                                      # another table names it too
    check(copied(cache), table, np.array([96, 70, 60]), "all ask")
    check(copied(cache), table, np.array([1, 0, 60]), "some ask")


@pytest.mark.parametrize("fmt,block,dim,shared", [("fp8", 32, 128, False), ("mxfp4", 32, 64, False), ("nvfp4", 16, 512, True)])
@pytest.mark.parametrize("release", [True, False])
def test_beams_with_pages_ahead(fmt, block, dim, shared, release):
    """A generation reserved ahead, a tree drafted and accepted up to a page's end, forks, rows appended by every beam:
    each beam's context is kept apart from any table, as a list of rows, and attention has to read that."""
    g = np.random.default_rng(dim)
    size, heads, T, lengths = 16, 2, 6, [45, 16, 3]
    cache = pools(g, 120, heads, size, dim, fmt, block, shared)
    table = counted(table_of(g, lengths, size, 9, 120), lengths, 120)
    kinds = ("k",) if shared else ("k", "v")
    kept = []                                            # of each sequence: (codes, scales) of every position, by pool
    for b, n in enumerate(lengths):
        at = [(table[0][b, p // size], p % size) for p in range(n)]
        kept.append([{name: cache[name][p, :, r].copy() for name in paged.POOLS if cache[name] is not None} for p, r in at])
    gpu, at = on_gpu(cache), table_on_gpu(table)

    def write(n):
        """n rows of every sequence appended on the card; what each position then holds."""
        B, out = at.pages.shape[0], []
        x = {name: values(g, (B, n, heads, dim), "bf16") for name in kinds}
        mxq.cache_append(gpu, at, x["k"].to(dev()), x["v"].to(dev()) if "v" in x else None)
        packed = {name: oracle.quantize_cache_packed(f64(x[name]), fmt, block) for name in kinds}
        for b in range(B):
            out.append([{f"{name}_{part}": packed[name][i][b, j] for name in kinds for i, part in enumerate(("codes", "scales"))}
                        for j in range(n)])
        return out

    def attends(T, what, rows):
        """Attention on the card against a cache of the kept rows alone, in pages of their own."""
        B, n = len(rows), max(len(r) for r in rows)
        W = -(-n // size)
        plain = dict(fmt=fmt, block=block, **{name: None for name in paged.POOLS})
        for name in rows[0][0]:
            plain[name] = np.zeros((B * W, *cache[name].shape[1:]), np.uint8)
            for b, seq in enumerate(rows):
                for p, row in enumerate(seq):
                    plain[name][b * W + p // size, :, p % size] = row[name]
        own = counted(np.arange(B * W, dtype=np.int32).reshape(B, W), [len(r) - T for r in rows], B * W)
        check_attention(values(g, (B, T, 4, dim), "bf16"), plain, own, what, (gpu, at))

    at, short = mxq.cache_reserve(gpu, at, 64)           # the whole generation
    assert short.tolist() == [0] * 3
    drafted = write(T)
    attends(T, "drafted", [k + d for k, d in zip(kept, drafted)])
    accepted = [[0, 3, 5], [1], [0, 1, 2]]
    at = mxq.cache_accept(gpu, at, i32([a + [-1] * (3 - len(a)) for a in accepted]))
    kept = [k + [d[i] for i in a] for k, d, a in zip(kept, drafted, accepted)]
    assert at.lengths.tolist() == [48, 17, 6]
    for step, parents in enumerate(([0, 0, 2, 2, 1], [1, 0, 0, 3, 4, 4], [5, 4, 0, 1, 1, 2, 2])):
        old = at
        at = mxq.cache_fork(at, i32(parents), release=release)
        if not release:                                  # the table before is given up after it
            gone = mxq.cache_free(gpu, old._replace(refs=at.refs))
            at = at._replace(refs=gone.refs)
        at, short = mxq.cache_reserve(gpu, at, 17)       # more than a page ahead
        assert short.tolist() == [0] * len(parents)
        held_alone(at, short.tolist(), at.lengths.cpu().numpy(), [17] * len(parents), size)
        new = write(3)
        kept = [kept[p] + new[b] for b, p in enumerate(parents)]
        attends(3, f"beams of step {step}", kept)
        at = at._replace(lengths=at.lengths + 3)
    at = mxq.cache_compact(gpu, at)
    q_rows = kept
    at = at._replace(lengths=at.lengths - 1)
    attends(1, "compacted", q_rows)


def test_a_captured_reserve_of_shared_pages():
    """Two graphs whose reserves have counts of shared pages in their workspaces, replayed in turn with eager calls between."""
    made = []
    for seed in range(2):
        g = np.random.default_rng(seed)
        cache = pools(g, 200, 1, 16, 64, "fp8", 32)
        tables = [table_ahead(g, 20, 6, 16, 200, 3) for _ in range(3)]
        tokens = i32(g.integers(0, 40, 20))
        static = on_gpu(cache), table_on_gpu(tables[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            mxq.cache_reserve(on_gpu(cache), static[1], tokens)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = mxq.cache_reserve(*static, tokens)
        made.append((cache, tables, tokens, static, graph, outs))
    for turn in range(6):
        for cache, tables, tokens, static, graph, outs in made:
            for pool, name in zip(static[0], paged.POOLS):
                pool.copy_(torch.from_numpy(cache[name]))
            for t, a in zip(static[1], tables[turn % 3]):
                t.copy_(torch.from_numpy(a))
            graph.replay()
            fresh = on_gpu(cache)
            want, lack = mxq.cache_reserve(fresh, static[1], tokens)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[0], want)) and torch.equal(outs[1], lack), turn
            assert all(torch.equal(a, b) for a, b in zip(static[0][:4], fresh[:4])), turn
