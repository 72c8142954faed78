"""The attention kernels' integer rules at the ends of their ranges (compiled for the CPU, no GPU needed)."""
import ctypes
import itertools
import os
import subprocess

import pytest

from tests.test_kv4_index_cpu import L as rules  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("kv4") / "kv4_index_ends.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC",
                    os.path.join(HERE, "native", "kv4_index_ends.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def seen_range(n, m, i, causal, window):
    """Keys [lo, hi) of query i of m, in whole numbers without a range."""
    hi = max(0, n - m + i + 1) if causal else n
    lo = max(0, n - m + i + 1 - window) if window else 0
    return lo, hi


WINDOWS = [0, 1, 63, 1024, 2 ** 30, TOP - 200, TOP - 1, TOP]


@pytest.mark.parametrize("keys", [32, 64])
def test_windows_up_to_the_largest_number(L, keys):
    """Also where queries stand before the first key, so that p + 1 - window lies below -2^31."""
    out = (ctypes.c_int * 2)()
    for n, m, window in itertools.product([0, 1, 5, 64, 1000, 1 << 30], [1, 2, 5, 200, 70000], WINDOWS):
        L.steps(m, n, 1, window, keys, out)
        first, count = out
        for i in sorted({0, 1, m // 2, m - 2, m - 1} & set(range(m))):
            lo, hi = seen_range(n, m, i, True, window)
            assert (L.lo(n, m, i, window), L.hi(n, m, i, 1)) == (lo, hi), (n, m, i, window)
            if lo < hi:
                assert keys * first <= lo and hi <= keys * (first + count)
        assert first >= 0 and count >= 1 and keys * first <= max(0, n)


def test_a_tiles_parts_cover_its_keys_once(L):
    """Every step that a query of the tile sees is in one of its parts, and all of them lie among the cuts."""
    out, sp = (ctypes.c_int * 4)(), (ctypes.c_int * 2)()
    for n, m, window, cuts in itertools.product([0, 1, 70, 1000, 5000], [1, 33, 200, 6000], WINDOWS, [1, 2, 3, 8]):
        for causal in ([1] if window else [0, 1]):
            L.steps(m, n, causal, window, 64, sp)
            first, count = sp
            if cuts > count:
                continue
            for i0 in {0, m // 2, max(0, m - 32)}:
                i1 = min(m - 1, i0 + 31)
                los, his = zip(*(seen_range(n, m, i, causal, window) for i in (i0, i1)))
                want = set(range(min(los) // 64, -(-max(his) // 64)))
                got = []
                for part in range(cuts):
                    L.tile_part(m, n, causal, window, 64, i0, i1, cuts, part, out)
                    part0, parts, s0, s1 = out
                    assert 0 <= part0 and parts >= 1 and part0 + parts <= cuts, (n, m, window, cuts, i0)
                    if part0 <= part < part0 + parts:
                        got += range(s0, s1)
                assert sorted(got) == sorted(want) and all(s <= max(0, n - 1) // 64 for s in got)


def test_queries_past_max_q_do_not_move_the_others(L):
    out = (ctypes.c_int * 6)()
    for n, q, max_q, window, causal in itertools.product([0, 3, 100, 1 << 30], [1, 6, 200], [1, 4, 6, 1000], [0, 2, 50, TOP],
                                                         [0, 1]):
        if window and not causal:
            continue
        kept = min(q, max_q)
        for i in {0, kept // 2, kept - 1}:
            L.cut_and_see(3, 3 + q, n, 500, max_q, 1 << 30, i, causal, window, out)
            lo, hi = seen_range(n, q, i, causal, window)
            assert tuple(out[:4]) == (3, kept, lo, hi)
            if lo < hi:
                assert 32 * out[4] <= lo and hi <= 32 * (out[4] + out[5])
    L.cut_and_see(0, TOP, 5, TOP, 1, 64, 0, 1, TOP, out)
    assert tuple(out[:4]) == (0, 1, 0, 0)                       # far before the first key


def test_parts_are_few_more_than_pairs(rules):
    """What the workspace holds slots for, whatever the lengths are."""
    more = rules.parts_more()
    for B, heads, most in itertools.product([1, 3, 200], [1, 8, 40], [0, 1000, 5000, 1 << 20, 1 << 30]):
        steps = [max(1, -(-most // 32))] * B
        limit = rules.part_limit(heads * sum(steps), max(steps), 32)
        assert heads * sum(-(-n // limit) for n in steps) <= B * heads + more
        assert rules.decode_grid(B, heads, most) <= B * heads + more
