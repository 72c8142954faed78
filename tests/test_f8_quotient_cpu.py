"""The division-free quotient of fp32 values (the gated product's and the norm's codes), compiled for the host."""
import ctypes
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

from tests import f8_util as f

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "native", "f8_quotient_shim.cpp")


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("shim") / "f8_quotient_shim.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fno-fast-math", "-ffp-contract=off", SRC,
                    "-o", so, "-lm"], check=True)
    L = ctypes.CDLL(so)
    L.shim_hard.argtypes = [ctypes.c_long, ctypes.c_long, ctypes.POINTER(ctypes.c_long)]
    L.shim_hard.restype = ctypes.c_long
    L.shim_quotients.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_long]
    L.shim_reciprocal.argtypes = [ctypes.c_float]
    L.shim_reciprocal.restype = ctypes.c_float
    return L


def test_every_pair_next_to_a_border(shim):
    """Beyond these pairs the corrected quotient cannot differ from the division (see f8_quotient)."""
    edges = [(1 << 23) + i * (1 << 23) // 64 for i in range(65)]

    def run(k):
        n = ctypes.c_long(0)
        return shim.shim_hard(edges[k], edges[k + 1], ctypes.byref(n)), n.value

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        got = list(ex.map(run, range(64)))
    assert sum(n for n, _ in got) == 0
    assert sum(n for _, n in got) > 150_000_000


def quotients(shim, x, s):
    out = [np.empty_like(x) for _ in range(3)]
    shim.shim_quotients(*(a.ctypes.data for a in (x, s, *out)), len(x))
    return out


def borders():
    """The middles between e4m3 codes and between int8 codes."""
    grid = f.decode(np.arange(127, dtype=np.uint8))
    return (grid[1:] + grid[:-1]) / 2, np.arange(127) + 0.5


@pytest.mark.parametrize("e", range(-126, -60, 6))
def test_small_scales(shim, e):
    """Values nearest to the borders between codes, at scales down to the smallest: the division's quotients
    from 2^-11 on, smaller below; without the lift not so where the residual underflows."""
    rng = np.random.default_rng(-e)
    off = 0
    for middles in borders():
        n = 1_000_000
        s = np.ldexp(1 + rng.random(n), e).astype(np.float32)
        x = (middles[rng.integers(0, len(middles), n)] * s.astype(np.float64)).astype(np.float32)
        lifted, plain, division = quotients(shim, x, s)
        seen = division >= 2.0 ** -11
        np.testing.assert_array_equal(lifted[seen], division[seen])
        assert (lifted[~seen] <= 2.0 ** -11).all()
        off += int((plain[seen] != division[seen]).sum())
    assert (off > 0) == (e <= -108)


def test_reciprocals(shim):
    for s in (1.0, 0.3, 2.0 ** -90, 1e30):
        assert shim.shim_reciprocal(s) == np.float32(1) / np.float32(s)
    below = float(np.nextafter(np.float32(2.0 ** -90), np.float32(0)))
    for s in (below, 2.0 ** -126):
        assert shim.shim_reciprocal(s) == -(np.float32(1) / (np.float32(s) * np.float32(2.0 ** 64)))
    assert shim.shim_reciprocal(0.0) == 0 and shim.shim_reciprocal(float("nan")) == 0
