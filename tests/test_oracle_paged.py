"""Pins of the paged cache's oracle: hand-worked tables, attention against a
dense softmax and its limits, and invariants of the counts."""

import numpy as np
import pytest

import oracle
from oracle import paged
from tests.paged_util import counted, copied, pools, table_of


def small(seed=0, size=16, heads=2, dim=64, pages=12, fmt="fp8", block=32, shared=False):
    g = np.random.default_rng(seed)
    return g, pools(g, pages, heads, size, dim, fmt, block, shared)


def test_hand_worked_fork_and_free():
    rows = np.array([[4, 1, -1], [2, 9, 3]], np.int32)          # page 9 is outside a pool of 6
    refs = np.array([0, 1, 1, 1, 1, 0], np.int32)
    new, n, held = paged.fork((rows, np.array([20, 40], np.int32), refs), [1, 1, 0, 7], 16)
    assert new.tolist() == [[2, -1, 3], [2, -1, 3], [4, 1, -1], [-1, -1, -1]]
    assert n.tolist() == [40, 40, 20, 0] and held.tolist() == [0, 2, 3, 3, 2, 0]
    new, n, held = paged.fork((rows, np.array([20, 40], np.int32), refs), [0, 1], 16, release=True, keep=[16, 99])
    assert new.tolist() == [[4, -1, -1], [2, -1, 3]] and n.tolist() == [16, 40]
    assert held.tolist() == [0, 0, 1, 1, 1, 0]


def test_hand_worked_reserve():
    _, cache = small(pages=8)
    # three sequences share page 5 (20 rows cached: 4 of its 16 filled); page 7 is all of the second page of none
    rows = np.array([[2, 5, -1], [2, 5, -1], [2, 5, -1]], np.int32)
    table = (rows, np.array([20, 20, 20], np.int32), np.array([0, 0, 3, 0, 1, 3, 0, 1], np.int32))
    before = copied(cache)
    (new, n, held), lack = paged.reserve(cache, table, [1, 1, 1])
    assert new.tolist() == [[2, 0, -1], [2, 1, -1], [2, 5, -1]] and lack.tolist() == [0, 0, 0]
    assert held.tolist() == [1, 1, 3, 0, 1, 1, 0, 1]
    for name in paged.POOLS:
        assert np.array_equal(cache[name][1, :, :4], before[name][5, :, :4])
        assert np.array_equal(cache[name][1, :, 4:], before[name][1, :, 4:])
    # 13 more positions need the third page too; the first asks for nothing
    (new, n, held), lack = paged.reserve(cache, table, [0, 13, 13])
    assert new.tolist() == [[2, 5, -1], [2, 0, 1], [2, 3, 6]] and lack.tolist() == [0, 0, 0] and held[5] == 1
    # 30 more: past the table's room
    (new, n, held), lack = paged.reserve(cache, table, [30, 30, 30])
    assert lack.tolist() == [1, 1, 1 + 1] and new.tolist() == [[2, 0, 1], [2, 3, 6], [2, 5, -1]]


def test_reserve_when_a_copy_fails():
    _, cache = small(pages=4)
    table = (np.array([[2], [2], [2]], np.int32), np.full(3, 5, np.int32), np.array([0, 1, 3, 1], np.int32))
    (new, _, held), lack = paged.reserve(cache, table, [1, 1, 1])
    # the one free page goes to the first; the second and the third are left together
    assert new.tolist() == [[0], [2], [2]] and lack.tolist() == [0, 1, 1] and held.tolist() == [1, 1, 2, 1]


def test_hand_worked_accept_and_compact():
    g, cache = small(pages=6)
    rows = np.array([[3, 1, 4]], np.int32)
    table = counted(rows, [14], 6)
    before = copied(cache)
    _, n, _ = paged.accept(cache, table, np.array([[0, 2, 3, 9, -1]], np.int32))
    assert n.tolist() == [18]
    where = lambda p: (rows[0, p // 16], p % 16)  # noqa: E731
    for a, d in enumerate([0, 2, 3, 9]):
        (i, x), (j, y) = where(14 + a), where(14 + d)
        assert np.array_equal(cache["k_codes"][i, :, x], before["k_codes"][j, :, y])
    for bad, count in ([[1, 1, 2]], 1), ([[3, 2]], 1), ([[-1, 2]], 0), ([[0, 1, 40]], 2):
        assert paged.accept(copied(before), table, np.array(bad, np.int32))[1].tolist() == [14 + count]
    table = counted(np.array([[5, 2, -1], [5, -1, 9]], np.int32), [20, 9], 6)
    cache = copied(before)
    new, n, held = paged.compact(cache, table)
    assert new.tolist() == [[1, 0, -1], [1, -1, -1]] and held.tolist() == [1, 2, 0, 0, 0, 0]
    assert np.array_equal(cache["v_codes"][0], before["v_codes"][2])
    assert np.array_equal(cache["v_scales"][1], before["v_scales"][5])


@pytest.mark.parametrize("fmt,block", [("fp8", 64), ("mxfp4", 32), ("nvfp4", 16)])
def test_append_is_quantize_cache_packed(fmt, block):
    g, cache = small(3, fmt=fmt, block=block)
    table = counted(table_of(g, [40, 20], 16, 3, 12), [17, 0], 12)
    x = g.standard_normal((2, 20, 2, 64))
    paged.append(cache, table, x, -x, counts=np.array([20, 3], np.int32))
    codes, scales = oracle.quantize_cache_packed(x, fmt, block)
    for b, n, m in ((0, 17, 20), (1, 0, 3)):
        for j in range(m):
            page, row = table[0][b, (n + j) // 16], (n + j) % 16
            assert np.array_equal(cache["k_codes"][page, :, row], codes[b, j])
            assert np.array_equal(cache["v_scales"][page, :, row], scales[b, j])


def test_append_leaves_shared_and_missing_pages():
    g, cache = small(4)
    rows = np.array([[3, -1], [3, 5]], np.int32)
    table = counted(rows, [14, 14], 12)
    before = copied(cache)
    paged.append(cache, table, g.standard_normal((2, 4, 2, 64)), g.standard_normal((2, 4, 2, 64)))
    assert np.array_equal(cache["k_codes"][3], before["k_codes"][3])
    assert not np.array_equal(cache["k_codes"][5, :, :2], before["k_codes"][5, :, :2])


def test_attention_against_a_dense_softmax():
    g, cache = small(5, fmt="mxfp4")
    lengths, T = [30, 0, 5], 3
    table = counted(table_of(g, [33, 3, 8], 16, 3, 12), lengths, 12)
    q = g.standard_normal((3, T, 4, 64))
    tree = np.tril(np.ones((3, T, T), bool))
    tree[:, 2, 1] = False
    out, lse, _, _, _, met = paged.attention(q, cache, table, mask=tree)
    for b, n in enumerate(lengths):
        k = np.concatenate([paged._values(cache["k_codes"][p], cache["k_scales"][p], cache)
                            for p in table[0][b] if p >= 0], 1)[:, : n + T]
        v = np.concatenate([paged._values(cache["v_codes"][p], cache["v_scales"][p], cache)
                            for p in table[0][b] if p >= 0], 1)[:, : n + T]
        for i in range(T):
            for h in range(4):
                s = k[h // 2] @ q[b, i, h] / 8.0
                s[n:] = np.where(tree[b, i], s[n:], -np.inf)
                e = np.exp(s - s.max())
                assert np.allclose(out[b, i, h], e @ v[h // 2] / e.sum(), rtol=1e-12, atol=1e-14)
                assert np.isclose(lse[b, i, h], np.log(np.exp(s).sum()))
                assert met[b, i, h] == n + tree[b, i].sum()


def test_attention_limits():
    g, cache = small(6)
    table = counted(np.array([[7, -1, 2], [-1, -1, -1]], np.int32), [40, 20], 12)
    q = np.zeros((2, 2, 2, 64))
    out, lse, _, _, _, met = paged.attention(q, cache, table, counts=np.array([1, 2], np.int32))
    # equal weights: the mean of the rows that exist (16 of the first page, 9 of the third)
    v = paged._values(cache["v_codes"], cache["v_scales"], cache)
    want = np.concatenate([v[7], v[2][:, :9]], 1).mean(1)
    assert np.allclose(out[0, 0], want) and np.allclose(lse[0, 0], np.log(25)) and met[0, 0, 0] == 25
    assert not out[0, 1].any() and not out[1].any() and np.isneginf(lse[1]).all()     # padding, and no page at all
    # a large scale: the best row
    q = g.standard_normal((2, 2, 2, 64))
    out = paged.attention(q, cache, table, scale=1e6)[0]
    k = paged._values(cache["k_codes"], cache["k_scales"], cache)
    s = np.concatenate([k[7], k[2][:, :9]], 1)[0] @ q[0, 0, 0]
    assert np.allclose(out[0, 0, 0], np.concatenate([v[7], v[2][:, :9]], 1)[0, s.argmax()])


def test_counts_stay_whole():
    """Forks, frees and reserves in any order: every page is named refs times, and no free page is named."""
    g, cache = small(7, pages=40)
    table = counted(table_of(g, [20, 35, 9], 16, 6, 40), [20, 35, 9], 40)
    for step in range(30):
        kind = g.integers(3)
        B = len(table[0])
        if kind == 0:
            table = paged.fork(table, g.integers(0, B, g.integers(1, 6)), 16, release=True)
        elif kind == 1:
            table = paged.fork(table, list(range(B)), 16, release=True, keep=g.integers(0, 60, B))
        else:
            table, lack = paged.reserve(cache, table, g.integers(0, 20, B))
        assert np.array_equal(table[2], paged._count(table[0], 40)), (step, kind)
    moved = paged.compact(cache, table)
    n = int((table[2] > 0).sum())
    assert (moved[2][:n] > 0).all() and not moved[2][n:].any() and np.array_equal(moved[2], paged._count(moved[0], 40))
