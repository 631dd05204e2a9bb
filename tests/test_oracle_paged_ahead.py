"""Pins of the oracle's cache_reserve where pages were reserved ahead and are
shared: entries past the cached positions that other sequences name too."""

import numpy as np
import pytest

import oracle
from oracle import paged
from tests.paged_util import copied, counted, pools, table_of


def held_alone(cache, table, tokens, lack):
    """Each entry of the next positions of a sequence that lacks nothing names a page of its own."""
    pages, lengths, refs = table
    size = cache["k_codes"].shape[2]
    for b, n in enumerate(lengths):
        if tokens[b] > 0 and lack[b] == 0:
            for slot in range(n // size, -(-(int(n) + int(tokens[b])) // size)):
                assert 0 <= pages[b, slot] < len(refs) and refs[pages[b, slot]] == 1, (b, slot)


def written(cache, table, k, b, n):
    """Whether rows k of sequence b lie at its positions n, n + 1, ..."""
    codes, scales = oracle.quantize_cache_packed(k, cache["fmt"], cache["block"])
    for j in range(len(k)):
        page, row = paged._place(cache, table[0][b], n + j)
        if not (np.array_equal(cache["k_codes"][page, :, row], codes[j])
                and np.array_equal(cache["k_scales"][page, :, row], scales[j])):
            return False
    return True


def test_hand_worked_pages_ahead():
    g = np.random.default_rng(0)
    cache = pools(g, 10, 2, 16, 64, "fp8", 32)
    # two sequences of 20 rows share their pages, one of them (7) behind the rows; page 8 holds positions of a third
    rows = np.array([[2, 5, 7, -1], [2, 5, 7, -1], [8, 7, -1, -1]], np.int32)
    table = counted(rows, [20, 20, 16], 10)
    assert table[2].tolist() == [0, 0, 2, 0, 0, 2, 0, 3, 1, 0]
    before = copied(cache)
    # page 5 is copied for the first and left to the second; of page 7 the first and the second get others, the third,
    # whose position 16 it holds, keeps it
    (new, n, held), lack = paged.reserve(copied(cache), table, [20, 20, 1])
    assert new.tolist() == [[2, 0, 1, -1], [2, 5, 3, -1], [8, 7, -1, -1]] and lack.tolist() == [0, 0, 0]
    assert held.tolist() == [1, 1, 2, 1, 0, 1, 0, 1, 1, 0] and n.tolist() == [20, 20, 16]
    # only filled rows come along
    (new, _, held), _ = paged.reserve(cache, table, [20, 0, 0])
    assert new.tolist() == [[2, 0, 1, -1], [2, 5, 7, -1], [8, 7, -1, -1]] and held.tolist() == [1, 1, 2, 0, 0, 1, 0, 2, 1, 0]
    for name in paged.POOLS:
        assert np.array_equal(cache[name][0, :, :4], before[name][5, :, :4])
        assert np.array_equal(cache[name][0, :, 4:], before[name][0, :, 4:])
        assert np.array_equal(cache[name][1], before[name][1])


def test_pages_ahead_when_the_pool_runs_out():
    g = np.random.default_rng(1)
    cache = pools(g, 5, 1, 16, 64, "fp8", 32)
    rows = np.array([[0, 3], [1, 3], [2, 3]], np.int32)
    table = counted(rows, [16, 16, 16], 5)
    (new, _, held), lack = paged.reserve(cache, table, [1, 1, 1])
    assert new.tolist() == [[0, 4], [1, 3], [2, 3]] and lack.tolist() == [0, 1, 1] and held.tolist() == [1, 1, 1, 2, 1]


def test_the_same_page_twice_in_a_row():
    g = np.random.default_rng(2)
    cache = pools(g, 5, 1, 16, 64, "fp8", 32)
    table = counted(np.array([[0, 3, 3]], np.int32), [16], 5)
    (new, _, held), lack = paged.reserve(cache, table, [32])
    assert new.tolist() == [[0, 1, 3]] and lack.tolist() == [0] and held.tolist() == [1, 1, 0, 1, 0]


def test_rows_of_beams_with_a_page_ahead_are_written():
    """Drafted rows ahead, some of them accepted up to the end of a page, then two beams that each write a row."""
    g = np.random.default_rng(3)
    cache = pools(g, 12, 2, 16, 64, "mxfp4", 32)
    table = counted(table_of(g, [45], 16, 6, 12), [45], 12)
    table, lack = paged.reserve(cache, table, [6])
    table = paged.accept(cache, table, np.array([[0, 1, 2]], np.int32))
    assert table[1].tolist() == [48] and table[0][0, 3] >= 0
    table = paged.fork(table, [0, 0], 16, release=True)
    table, lack = paged.reserve(cache, table, [1, 1])
    assert lack.tolist() == [0, 0]
    held_alone(cache, table, [1, 1], lack)
    k, v = g.standard_normal((2, 1, 2, 64)), g.standard_normal((2, 1, 2, 64))
    paged.append(cache, table, k, v)
    assert written(cache, table, k[0], 0, 48) and written(cache, table, k[1], 1, 48)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("release", [True, False])
def test_what_lacks_nothing_can_be_written(seed, release):
    """Reserves, some far ahead, appends, accepts, forks and frees in any order."""
    g = np.random.default_rng(seed)
    size, total = 16, 60
    cache = pools(g, total, 1, size, 64, "fp8", 64)
    table = counted(table_of(g, [20, 35, 9], size, 7, total), [20, 35, 9], total)
    met = 0
    for step in range(120):
        kind, B = g.integers(5), len(table[0])
        if kind == 0:
            new = paged.fork(table, g.integers(0, B, g.integers(1, 6)), size, release=True)
            if not release:             # the old table is given up afterwards
                new = paged.fork(table, g.integers(0, B, g.integers(1, 6)), size)
                new = new[0], new[1], (new[2] - paged._count(table[0], total)).astype(np.int32)
            table = new
        elif kind == 1:
            table = paged.fork(table, list(range(B)), size, release=True, keep=g.integers(0, 90, B))
        else:
            tokens = g.integers(0, 50, B) * (g.random(B) < 0.8)
            beyond = [p for row, n in zip(table[0], table[1]) for p in row[-(-int(n) // size):] if p >= 0]
            met += sum(table[2][p] > 1 for p in beyond)
            table, lack = paged.reserve(cache, table, tokens)
            held_alone(cache, table, tokens, lack)
            most = int(g.integers(1, 20))
            k = g.standard_normal((B, most, 1, 64))
            counts = np.minimum(tokens, most).astype(np.int32)
            paged.append(cache, table, k, k, counts)
            for b in range(B):
                if lack[b] == 0:
                    assert written(cache, table, k[b, : counts[b]], b, int(table[1][b]))
            accepted = np.full((B, 3), -1, np.int32)
            for b in range(B):
                if lack[b] == 0:
                    accepted[b, : min(3, counts[b])] = np.arange(min(3, counts[b]))
            table = paged.accept(cache, table, accepted)
        assert np.array_equal(table[2], paged._count(table[0], total)), (step, kind)
    assert met > 0                      # shared pages past the lengths were there
