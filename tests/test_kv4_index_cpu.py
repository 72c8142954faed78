"""The attention kernels' integer rules on hostile tables: whatever the entries are, every row, key and
page they lead to lies inside the call's buffers (compiled for the CPU, no GPU needed)."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
TOP, LOW = 2 ** 31 - 1, -2 ** 31


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("kv4") / "kv4_index.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "native", "kv4_index_shim.cpp"),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.part_limit.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    lib.tile_limit.argtypes = [ctypes.c_int64, ctypes.c_int]
    lib.tiles.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p]
    lib.decode_grid.restype = ctypes.c_int64
    lib.decode_grid.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    lib.page_ok.argtypes = [ctypes.c_int, ctypes.c_int64]
    return lib


def cut(L, *a):
    out = (ctypes.c_int * 3)()
    L.cut(*a, out)
    return tuple(out)


def test_cut_stays_inside(L):
    marks = [LOW, -7, -1, 0, 1, 5, 17, 1000, TOP]
    for start, end, n, T, max_q, most in itertools.product(marks, marks, marks, [1, 17, TOP], [1, 9], [0, 64, 1 << 30]):
        q0, m, keys = cut(L, start, end, n, T, min(max_q, T), most)
        assert 0 <= keys <= most and 0 <= m <= max_q and 0 <= q0 and q0 + m <= T, (start, end, n, T)


def test_cut_keeps_what_is_right(L):
    assert cut(L, 3, 9, 100, 20, 8, 128) == (3, 6, 100)
    assert cut(L, 3, 9, 100, 20, 4, 128) == (3, 4, 100)
    assert cut(L, 3, 3, 0, 20, 4, 128) == (3, 0, 0)


@pytest.mark.parametrize("keys", [32, 64])
def test_visible_ranges_and_steps(L, keys):
    """Every key that some query sees lies in the steps; there is always a step while there are queries."""
    out = (ctypes.c_int * 2)()
    for n, m, causal, window in itertools.product([0, 1, 31, 32, 33, 64, 100], [0, 1, 2, 31, 40, 150], [0, 1],
                                                  [0, 1, 7, 32, 99]):
        if window and not causal:
            continue
        L.steps(m, n, causal, window, keys, out)
        first, count = out
        assert (count == 0) == (m == 0) and first >= 0
        for i in range(m):
            lo, hi = L.lo(n, m, i, window), L.hi(n, m, i, causal)
            p = n - m + i
            seen = [j for j in range(n) if (not causal or j <= p) and (not window or j > p - window)]
            assert [j for j in range(n) if lo <= j < hi] == seen
            if seen:
                assert keys * first <= seen[0] and seen[-1] < keys * (first + count)
        assert keys * (first + count) <= -(-n // keys) * keys or count == 1


def test_steps_at_the_ends(L):
    out = (ctypes.c_int * 2)()
    L.steps(1, 1 << 30, 1, 0, 32, out)
    assert tuple(out) == (0, 1 << 25)
    L.steps(5, 1 << 30, 1, TOP, 32, out)
    assert tuple(out) == (0, 1 << 25)
    L.steps(TOP, 7, 1, 3, 64, out)
    assert out[0] == 0 and out[1] == 1


def test_parts_cover_the_steps_and_fit_the_grid(L):
    r = random.Random(1)
    for _ in range(600):
        keys = r.choice([32, 64])
        B, heads, most = r.randint(1, 70), r.randint(1, 40), 16 * r.choice([0, 1, 2, 60, 65, 5000, 1 << 20])
        counts = [max(1, -(-r.choice([most, r.randint(0, most)]) // keys)) if r.random() < 0.8 else 0 for _ in range(B)]
        limit = L.part_limit(heads * sum(counts), max(counts), keys)
        parts = [-(-n // limit) for n in counts]
        assert heads * sum(parts) <= L.decode_grid(B, heads, most)
        assert max(parts) <= 64                                    # arrivals are counted in 16 bits
        for n, k in zip(counts, parts):
            if n:
                cuts = [L.split(n, k, i) for i in range(k + 1)]
                assert cuts[0] == 0 and cuts[-1] == n
                assert all(0 < b - a <= limit for a, b in zip(cuts, cuts[1:]))


def test_parts_at_the_ends(L):
    assert L.part_limit(0, 0, 32) == 32 and L.part_limit(0, 0, 64) == 16 and L.part_limit(1 << 60, 5, 64) == 0x3fffffff
    assert L.split(1 << 25, 1025, 1025) == 1 << 25


def test_tiles_fit_the_grid_and_the_slots(L):
    """The kernel for many rows: workgroups for every part, and a slot for every part of a cut item."""
    r = random.Random(2)
    out = (ctypes.c_int64 * 3)()
    for _ in range(600):
        B, heads, group, most = r.randint(1, 70), r.randint(1, 9), r.randint(1, 9), 16 * r.choice([1, 20, 300, 70000])
        m = [r.randint(0, 700) for _ in range(B)]
        T = sum(m)
        if not T:
            continue
        L.tiles(T, B, group, heads, most, out)
        grid, slots, rows = out
        tiles = [-(-q * group // rows) for q in m]
        steps = [max(1, -(-r.choice([most, r.randint(0, most)]) // 64)) if q else 0 for q in m]
        limit = L.tile_limit(heads * sum(t * s for t, s in zip(tiles, steps)), 64)
        cuts = [-(-s // limit) for s in steps]
        assert heads * sum(t * k for t, k in zip(tiles, cuts)) <= grid
        assert heads * sum(t * k for t, k in zip(tiles, cuts) if k > 1) <= slots
        assert max(cuts) < 65536


def test_pages(L):
    assert L.page_ok(0, 1) and L.page_ok(6, 7)
    for page, pages in [(-1, 7), (7, 7), (TOP, 7), (LOW, 7)]:
        assert not L.page_ok(page, pages)
