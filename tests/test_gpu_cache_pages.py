"""GPU parity of the cache's page operations against the CPU oracle: tables,
lengths, counts and every byte of the pools, for forks, frees, reserves with
copies of shared pages, accepted drafts and compaction; odd sizes, tables and
lengths that name nothing, pools that run out."""

import numpy as np
import pytest
import torch

import nvfp4_quantization_grouped_amd as mxq
from oracle import paged
from tests.gpu_util import dev
from tests.paged_util import assert_same_pools, assert_same_table, copied, counted, on_gpu, pools, table_of, table_on_gpu

pytestmark = pytest.mark.gpu

i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev())  # noqa: E731


def random_table(g, B, W, size, pages, longest=None):
    """Sequences that share some of their pages, in a pool where some are free."""
    lengths = g.integers(0, (longest or W * size) + 1, B)
    rows = np.full((B, W), -1, np.int32)
    order = list(g.permutation(pages))
    for b in range(B):
        for i in range(-(-lengths[b] // size)):
            if b and rows[b - 1, i] >= 0 and g.random() < 0.5:
                rows[b, i] = rows[b - 1, i]
            elif order:
                rows[b, i] = order.pop()
    return counted(rows, lengths, pages)


def check_reserve(cache, table, tokens, what):
    gpu = on_gpu(cache)
    each = tokens if isinstance(tokens, int) else i32(tokens)
    got, lack = mxq.cache_reserve(gpu, table_on_gpu(table), each)
    want, want_lack = paged.reserve(cache, table, [tokens] * len(table[0]) if isinstance(tokens, int) else tokens)
    assert_same_table(got, want, what)
    assert np.array_equal(lack.cpu().numpy(), want_lack), f"{what}: {lack.tolist()} {want_lack.tolist()}"
    assert_same_pools(gpu, cache, what)


@pytest.mark.parametrize("B,C,W,pages", [(1, 1, 1, 1), (3, 5, 4, 20), (64, 64, 9, 300), (5, 130, 70, 200), (7, 3, 33, 5000)])
@pytest.mark.parametrize("release", [False, True])
def test_fork(B, C, W, pages, release):
    g = np.random.default_rng(B + C)
    table = random_table(g, B, W, 16, pages)
    parents = g.integers(-1, B + 1, C)                           # some of nobody
    got = mxq.cache_fork(table_on_gpu(table), i32(parents), release=release)
    assert_same_table(got, paged.fork(table, parents, 16, release), "fork")


@pytest.mark.parametrize("B,W,pages,size", [(1, 1, 1, 16), (9, 5, 60, 64), (130, 17, 900, 256)])
def test_free(B, W, pages, size):
    g = np.random.default_rng(B)
    cache = pools(g, pages, 1, size, 64, "fp8", 64, True) if pages < 100 else None
    gpu = on_gpu(cache) if cache else mxq.paged_cache(pages, size, 1, 64, "fp8", 64, shared=True)
    table = random_table(g, B, W, size, pages)
    keep = g.integers(-3, W * size + 9, B)
    got = mxq.cache_free(gpu, table_on_gpu(table), i32(keep))
    assert_same_table(got, paged.fork(table, range(B), size, True, keep), "free")
    got = mxq.cache_free(gpu, table_on_gpu(table))
    assert int(got.pages.max()) == -1 and not got.lengths.any() and not got.refs.any()


@pytest.mark.parametrize("B,W,pages", [(600, 9, 2000), (455, 9, 3000), (456, 9, 3000), (40, 100, 70000)])
def test_free_and_fork_of_many_entries(B, W, pages):
    """Around the number of entries from which two launches take the place of one."""
    g = np.random.default_rng(B)
    gpu = mxq.paged_cache(pages, 32, 1, 64, "fp8", 64, shared=True)
    table = random_table(g, B, W, 32, pages)
    keep = g.integers(-3, W * 32 + 9, B)
    got = mxq.cache_free(gpu, table_on_gpu(table), i32(keep))
    assert_same_table(got, paged.fork(table, range(B), 32, True, keep), "free")
    parents = g.integers(0, B, B)
    got = mxq.cache_fork(table_on_gpu(table), i32(parents), release=True)
    assert_same_table(got, paged.fork(table, parents, 16, True), "fork")


def test_fork_of_entries_that_name_no_page():
    rows = np.array([[2, 5, -9], [1 << 30, 0, 2]], np.int32)
    table = rows, np.array([-4, 2 ** 31 - 1], np.int32), np.array([1, 0, 2, 0, 0], np.int32)
    got = mxq.cache_fork(table_on_gpu(table), i32([1, 0, 1]))
    assert_same_table(got, paged.fork(table, [1, 0, 1], 16), "entries")
    none = mxq.cache_fork(table_on_gpu(table), i32([]), release=True)
    assert none.pages.shape == (0, 3) and none.refs.tolist() == [0, 0, 0, 0, 0]


@pytest.mark.parametrize("B,W,size,pages", [
    (1, 1, 16, 2), (3, 4, 16, 30), (17, 3, 32, 90), (64, 6, 64, 500), (70, 80, 16, 6000), (1100, 2, 16, 3000)])
@pytest.mark.parametrize("seed", [0, 1])
def test_reserve(B, W, size, pages, seed):
    g = np.random.default_rng(1000 * seed + B)
    fmt, block = [("fp8", 64), ("nvfp4", 16)][seed]
    cache = pools(g, pages, 1 if pages > 400 else 3, size, 64, fmt, block, pages > 400)
    table = random_table(g, B, W, size, pages, W * size - 8)
    check_reserve(cache, table, g.integers(-2, size + 9, B), "reserve")


def test_reserve_one_token_for_all_and_long_prompts():
    g = np.random.default_rng(3)
    cache = pools(g, 700, 1, 16, 64, "mxfp4", 32)
    table = random_table(g, 20, 150, 16, 700, 300)
    check_reserve(copied(cache), table, 1, "one token")
    check_reserve(copied(cache), table, 0, "no token")
    check_reserve(copied(cache), table, g.integers(0, 2, 20) * 2100, "long prompts")       # 131 pages: two ballots


@pytest.mark.parametrize("free", [0, 1, 2, 3, 7])
def test_reserve_when_the_pool_runs_out(free):
    g = np.random.default_rng(free)
    pages, size = 40, 16
    cache = pools(g, pages, 2, size, 64, "fp8", 32)
    rows = np.full((9, 4), -1, np.int32)
    rows[:, 0], rows[:6, 1], rows[6:, 1] = 3, 4, 5
    table = counted(rows, [20] * 6 + [27] * 3, pages)
    refs = table[2]
    open_pages = np.flatnonzero(refs == 0)
    refs[open_pages[free:]] = 1                          # held by somebody else
    check_reserve(cache, (rows, table[1], refs), g.integers(0, 30, 9), "short of pages")


def test_reserve_past_the_table_and_odd_lengths():
    g = np.random.default_rng(5)
    cache = pools(g, 12, 1, 16, 64, "fp8", 32)
    rows = np.array([[0, 1], [2, -1], [99, -5], [-1, -1]], np.int32)
    table = rows, np.array([32, 2 ** 31 - 1, 7, -8], np.int32), np.array([1, 1, 1] + [0] * 6 + [-3, 0, 0], np.int32)
    check_reserve(cache, table, np.array([1, 5, 20, 2 ** 31 - 1], np.int64), "odd")


def test_reserve_with_many_pages():
    """More pages than one pass of the planning workgroup looks at, the free ones at the end."""
    g = np.random.default_rng(6)
    pages = 40000
    gpu = mxq.paged_cache(pages, 16, 1, 64, "nvfp4", 16, shared=True)
    rows, refs = np.full((50, 30), -1, np.int32), np.ones(pages, np.int32)
    rows[:, 0] = np.arange(50)
    refs[g.permutation(np.arange(30000, pages))[:1500]] = 0
    table = rows, np.full(50, 16, np.int32), refs
    got, lack = mxq.cache_reserve(gpu, table_on_gpu(table), 16 * 29)
    stub = {n: None for n in paged.POOLS}
    stub.update(fmt="nvfp4", block=16, k_codes=np.zeros((pages, 1, 16, 0), np.uint8))
    want, want_lack = paged.reserve(stub, table, [16 * 29] * 50)
    assert_same_table(got, want, "many pages")
    assert not want_lack.any() and not lack.any()


def test_reserve_without_sequences():
    gpu = mxq.paged_cache(5, 16, 1, 64, "fp8", 32)
    table = mxq.page_table(0, 3, gpu)._replace(refs=i32([1, 0, 2, 0, 0]))
    got, lack = mxq.cache_reserve(gpu, table, 4)
    assert got.refs.tolist() == [1, 0, 2, 0, 0] and lack.shape == (0,)


def paths(g, B, most, T):
    out = np.full((B, most), -1, np.int32)
    for b in range(B):
        path = np.sort(g.permutation(T)[: g.integers(0, min(most, T) + 1)])
        out[b, : len(path)] = path
    return out


@pytest.mark.parametrize("fmt,block,dim,shared", [
    ("fp8", 128, 128, False), ("fp8", 16, 512, False), ("mxfp4", 64, 64, True), ("nvfp4", 16, 64, False),
    ("nvfp4", 16, 512, True), ("mxfp4", 128, 256, False)])
@pytest.mark.parametrize("most,T", [(1, 1), (5, 9), (64, 64), (40, 100)])
def test_accept(fmt, block, dim, shared, most, T):
    g = np.random.default_rng(dim + most)
    lengths = [0, 15, 16, 30, 47]
    cache = pools(g, 50, 3, 16, dim, fmt, block, shared)
    table = counted(table_of(g, [n + T for n in lengths], 16, 11, 50), lengths, 50)
    accepted = paths(g, 5, most, T)
    gpu = on_gpu(cache)
    got = mxq.cache_accept(gpu, table_on_gpu(table), i32(accepted))
    assert_same_table(got, paged.accept(cache, table, accepted), "accept")
    assert_same_pools(gpu, cache, "accept")


def test_accept_ends_its_list():
    g = np.random.default_rng(0)
    cache = pools(g, 12, 2, 16, 64, "fp8", 64)
    rows = np.array([[0, 1], [2, 3], [4, -1], [5, 6], [7, 8], [9, 99], [10, 11]], np.int32)
    table = counted(rows, [10, 10, 10, 10, 30, 14, -9], 12)
    table[2][6] = 2                                              # shared
    accepted = np.array([[0, 2, 2, 3], [1, 5, 3, 9], [1, 2, 8, 9], [3, 4, 5, 8], [0, 1, 2, 3], [1, 2, 3, 4],
                         [2 ** 31 - 1, 1, 2, 3]], np.int32)
    gpu = on_gpu(cache)
    got = mxq.cache_accept(gpu, table_on_gpu(table), i32(accepted))
    assert_same_table(got, paged.accept(cache, table, accepted), "accept")
    assert_same_pools(gpu, cache, "accept")
    got = mxq.cache_accept(gpu, table_on_gpu(table), i32(np.zeros((7, 0))))
    assert got.lengths.tolist() == [10, 10, 10, 10, 30, 14, 0]


@pytest.mark.parametrize("pages,size,heads,dim,fmt,block,shared", [
    (1, 16, 1, 64, "fp8", 64, True), (2, 16, 1, 64, "nvfp4", 16, False), (37, 32, 3, 128, "mxfp4", 32, False),
    (200, 64, 2, 128, "fp8", 128, False), (90, 16, 1, 512, "fp8", 16, True)])
@pytest.mark.parametrize("share", [0.1, 0.5, 0.9])
def test_compact(pages, size, heads, dim, fmt, block, shared, share):
    g = np.random.default_rng(pages)
    cache = pools(g, pages, heads, size, dim, fmt, block, shared)
    used = np.flatnonzero(g.random(pages) < share)
    rows = np.full((6, max(1, len(used))), -1, np.int32)
    for p in used:
        for b in g.permutation(6)[: g.integers(1, 3)]:
            rows[b, g.integers(0, rows.shape[1])] = p
    table = counted(rows, g.integers(0, 9, 6), pages)
    gpu = on_gpu(cache)
    got = mxq.cache_compact(gpu, table_on_gpu(table))
    assert_same_table(got, paged.compact(cache, table), "compact")
    assert_same_pools(gpu, cache, "compact")


def test_compact_of_many_pages_and_odd_entries():
    g = np.random.default_rng(1)
    pages = 50001
    gpu = mxq.paged_cache(pages, 16, 1, 64, "nvfp4", 16, shared=True)
    refs = (g.random(pages) < 0.4).astype(np.int32) * g.integers(-1, 4, pages).astype(np.int32)
    rows = g.integers(-2, pages + 2, (20, 900)).astype(np.int32)
    mark = torch.arange(pages, device=dev())
    gpu.k_codes[:, 0, 0, :4] = (mark[:, None] >> torch.tensor([0, 8, 16, 24], device=dev()) & 255).to(torch.uint8)
    table = rows, np.zeros(20, np.int32), refs
    got = mxq.cache_compact(gpu, table_on_gpu(table))
    stub = {n: None for n in paged.POOLS}
    stub.update(fmt="nvfp4", block=16, k_codes=gpu.k_codes.cpu().numpy().copy())
    stub["k_codes"][:, 0, 0, :4] = (np.arange(pages)[:, None] >> np.array([0, 8, 16, 24]) & 255).astype(np.uint8)
    want = paged.compact(stub, table)
    assert_same_table(got, want, "compact")
    assert np.array_equal(gpu.k_codes.cpu().numpy(), stub["k_codes"])


def test_offsets_past_32_bits():
    """Rows copied, appended and moved in the last pages of a pool of 4.8 GB, all others of which are held."""
    pages, size, dim = 9300, 256, 512
    gpu = mxq.paged_cache(pages, size, 4, dim, "fp8", 128, shared=True)
    assert gpu.k_codes.numel() > 1 << 32
    g = np.random.default_rng(8)
    cache = pools(g, 6, 4, size, dim, "fp8", 128, True)
    far = np.array([8200, 8300, 8400, 9297, 9298, 9299])
    at = torch.from_numpy(far).to(dev())
    gpu.k_codes[at] = torch.from_numpy(cache["k_codes"]).to(dev())
    gpu.k_scales[at] = torch.from_numpy(cache["k_scales"]).to(dev())

    def placed(table):
        refs = np.ones(pages, np.int32)
        refs[far] = table[2]
        return np.where(table[0] >= 0, far[np.maximum(table[0], 0)], -1).astype(np.int32), table[1], refs

    def same(what):
        assert_same_table(on_card, placed(table), what)
        for name in ("k_codes", "k_scales"):
            assert np.array_equal(getattr(gpu, name)[at].cpu().numpy(), cache[name]), (what, name)
    table = counted(np.array([[5, -1], [5, -1], [4, -1]], np.int32), [200, 200, 250], 6)
    on_card, lack = mxq.cache_reserve(gpu, table_on_gpu(placed(table)), 9)
    table, want_lack = paged.reserve(cache, table, [9] * 3)
    assert lack.tolist() == want_lack.tolist() == [0, 0, 0]
    same("reserve")
    k = torch.from_numpy(g.standard_normal((3, 9, 4, dim)).astype(np.float32))
    mxq.cache_append(gpu, on_card, k.to(dev()))
    paged.append(cache, table, k.double().numpy())
    same("append")
    accepted = np.array([[1, 3, 8], [0, 1, -1], [2, 6, 7]], np.int32)
    on_card, table = mxq.cache_accept(gpu, on_card, i32(accepted)), paged.accept(cache, table, accepted)
    same("accept")


def test_refusals():
    gpu = mxq.paged_cache(6, 16, 2, 64, "fp8", 32)
    table = mxq.page_table(3, 2, gpu)
    for call, error in (
            (lambda: mxq.cache_fork(table, table.lengths.long()), TypeError),
            (lambda: mxq.cache_fork(table, table.pages), TypeError),
            (lambda: mxq.cache_free(gpu, table, table.lengths[:2]), TypeError),
            (lambda: mxq.cache_reserve(gpu, table, table.lengths.float()), TypeError),
            (lambda: mxq.cache_reserve(gpu, table._replace(pages=table.pages[0]), 1), TypeError),
            (lambda: mxq.cache_reserve(gpu, table._replace(refs=table.refs[1:]), 1), ValueError),
            (lambda: mxq.cache_reserve(gpu, table, 1 << 31), mxq.MxqError),
            (lambda: mxq.cache_reserve(gpu, mxq.page_table(4097, 1, gpu), 1), mxq.MxqError),
            (lambda: mxq.cache_accept(gpu, table, table.lengths), TypeError),
            (lambda: mxq.cache_accept(gpu, table, table.pages[:2]), TypeError),
            (lambda: mxq.cache_accept(gpu, table, i32(np.zeros((3, 65)))), mxq.MxqError),
            (lambda: mxq.cache_compact(gpu._replace(k_scales=gpu.k_scales[..., :1]), table), ValueError),
            (lambda: mxq.cache_fork(table, table.lengths.cpu()), ValueError)):
        with pytest.raises(error):
            call()
