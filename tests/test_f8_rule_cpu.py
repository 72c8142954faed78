"""The e4m3 rule's division-free quotient, compiled for the host, and the tests' own e4m3."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests import f8_util as f

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "native", "f8_rule_shim.cpp")


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("shim") / "f8_rule_shim.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fno-fast-math", "-ffp-contract=off", SRC,
                    "-o", so, "-lm"], check=True)
    L = ctypes.CDLL(so)
    L.shim_quotients.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_long)]
    L.shim_quotients.restype = ctypes.c_long
    L.shim_quotient.argtypes = [ctypes.c_float, ctypes.c_float]
    L.shim_quotient.restype = ctypes.c_float
    L.shim_scale.argtypes = [ctypes.c_float]
    L.shim_scale.restype = ctypes.c_float
    return L


def test_quotient_on_the_whole_domain(shim):
    """fl32(x / s) for every fp16 amax and every fp16 x up to it, without a division; the correction step
    is what makes it so."""
    from concurrent.futures import ThreadPoolExecutor
    top = 0x7C00
    edges = sorted({1, top, *(int(top * (i / 64) ** 0.5) for i in range(1, 64))})

    def run(k):
        n = ctypes.c_long(0)
        return shim.shim_quotients(edges[k], edges[k + 1], ctypes.byref(n)), n.value

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        got = list(ex.map(run, range(len(edges) - 1)))
    assert sum(n for n, _ in got) == 0
    assert sum(n for _, n in got) > 0


def test_zeros_keep_their_sign(shim):
    for s in (1.0, 0.3, 133.7, 2.0 ** -33):
        assert not np.signbit(shim.shim_quotient(0.0, s)) and np.signbit(shim.shim_quotient(-0.0, s))


def test_scale_of_tiny_blocks(shim):
    assert shim.shim_scale(448.0) == 1.0
    assert shim.shim_scale(0.0) == 0.0
    least = np.float32(2.0 ** -126 * 448)
    assert shim.shim_scale(float(least)) == 2.0 ** -126
    assert shim.shim_scale(float(np.nextafter(least, np.float32(0)))) in (0.0, 2.0 ** -126)
    assert shim.shim_scale(1e-40) == 0.0


def test_codes_of_the_tests():
    torch = pytest.importorskip("torch")
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(f.decode(np.arange(256, dtype=np.uint8)).astype(np.float32), every)
    rng = np.random.default_rng(5)
    grid = f.decode(np.arange(127, dtype=np.uint8))
    t = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(0, 1e-2, 4000), grid, -grid,
                        (grid[1:] + grid[:-1]) / 2, [-0.0]]).astype(np.float32)
    want = torch.from_numpy(t).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(f.encode(t), want)
