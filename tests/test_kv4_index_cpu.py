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
    lib.part_begin.restype = ctypes.c_int64
    lib.part_begin.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    lib.part_of.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    lib.parts.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
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


def test_visible_ranges_and_steps(L):
    """Every key that some query sees lies in the steps; there is always a step while there are queries."""
    out = (ctypes.c_int * 2)()
    for n, m, causal, window in itertools.product([0, 1, 31, 32, 33, 64, 100], [0, 1, 2, 31, 40, 150], [0, 1],
                                                  [0, 1, 7, 32, 99]):
        if window and not causal:
            continue
        L.steps(m, n, causal, window, out)
        first, count = out
        assert (count == 0) == (m == 0) and first >= 0
        for i in range(m):
            lo, hi = L.lo(n, m, i, window), L.hi(n, m, i, causal)
            p = n - m + i
            seen = [j for j in range(n) if (not causal or j <= p) and (not window or j > p - window)]
            assert [j for j in range(n) if lo <= j < hi] == seen
            if seen:
                assert 32 * first <= seen[0] and seen[-1] < 32 * (first + count)
        assert 32 * (first + count) <= (n + 31) // 32 * 32 or count == 1


def test_steps_at_the_ends(L):
    out = (ctypes.c_int * 2)()
    L.steps(1, 1 << 30, 1, 0, out)
    assert tuple(out) == (0, 1 << 25)
    L.steps(5, 1 << 30, 1, TOP, out)
    assert tuple(out) == (0, 1 << 25)
    L.steps(TOP, 7, 1, 3, out)
    assert out[0] == 0 and out[1] == 1


def test_parts_cover_the_units_once(L):
    r = random.Random(1)
    for _ in range(400):
        U, most, least = r.choice([1, 5, 37, 1000, 10 ** 6, 1 << 45]) + r.randint(0, 3), r.randint(1, 600), r.randint(1, 40)
        parts = L.parts(U, most, least)
        assert 1 <= parts <= most
        assert L.part_begin(U, parts, 0) == 0 and L.part_begin(U, parts, parts) == U
        for u in {0, U - 1, U // 2, r.randrange(U)}:
            i = L.part_of(U, parts, u)
            assert 0 <= i < parts and L.part_begin(U, parts, i) <= u < L.part_begin(U, parts, i + 1)


def test_pages(L):
    assert L.page_ok(0, 1) and L.page_ok(6, 7)
    for page, pages in [(-1, 7), (7, 7), (TOP, 7), (LOW, 7)]:
        assert not L.page_ok(page, pages)
