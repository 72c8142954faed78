"""How far the steps of the gated product's activation are from it in fp32, compiled for the host."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests.f8_activation import U, activation

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "native", "f8_activation_shim.cpp")


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("shim") / "f8_activation_shim.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fno-fast-math", "-ffp-contract=off", SRC,
                    "-o", so, "-lm"], check=True)
    L = ctypes.CDLL(so)
    L.shim_activation.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_long] + [ctypes.c_int] * 3

    def run(g, kind, exp_units=0, rcp_units=0):
        out = np.empty_like(g)
        L.shim_activation(g.ctypes.data, out.ctypes.data, len(g), kind != "silu", exp_units, rcp_units)
        return out
    return run


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("exp_units,rcp_units", [(0, 0), (1, 1), (1, -1), (-1, 1), (-1, -1)])
def test_bound(shim, kind, exp_units, rcp_units):
    rng = np.random.default_rng(7)
    g = np.concatenate([rng.uniform(-100, 100, 300_000), rng.uniform(-12, 12, 300_000), rng.normal(0, 1e-3, 50_000),
                        -np.exp2(rng.uniform(-130, 127, 50_000)), np.exp2(rng.uniform(-130, 127, 50_000))]).astype(np.float32)
    got = shim(g, kind, exp_units, rcp_units).astype(np.float64)
    want, bound = activation(g.astype(np.float64), kind)
    assert (np.abs(got - want) <= bound).all()


def test_the_size_of_it(shim):
    """With an ideal exponential and reciprocal: more than 2^-20 of the result from g = -20 on, and the bound
    within four times of what is seen."""
    rng = np.random.default_rng(8)
    for kind, low, least in (("silu", -30.0, 2.0 ** -19.5), ("silu", -60.0, 2.0 ** -18.5), ("gelu_tanh", -5.0, 2.0 ** -19)):
        g = rng.uniform(low, low * 0.9, 200_000).astype(np.float32)
        want, bound = activation(g.astype(np.float64), kind)
        off = np.abs(shim(g, kind).astype(np.float64) - want)
        assert (off / np.abs(want)).max() >= least
        assert (off / bound).max() >= 0.25
    g = rng.uniform(0, 60, 200_000).astype(np.float32)
    for kind in ("silu", "gelu_tanh"):
        want, bound = activation(g.astype(np.float64), kind)
        assert (bound <= 2.0 ** -20.9 * want + 2.0 ** -119).all() and bound.max() > 5 * U


def test_ends(shim):
    """Zeros keep their sign, large values are themselves, very negative ones -0, NaN stays."""
    g = np.array([0.0, -0.0, 100, 3e38, -100, -3e38, np.inf, np.nan], np.float32)
    for kind in ("silu", "gelu_tanh"):
        got = shim(g, kind)
        np.testing.assert_array_equal(got[[0, 1, 2, 3, 6]], g[[0, 1, 2, 3, 6]])
        assert not np.signbit(got[0]) and np.signbit(got[1]) and np.isnan(got[7])
        assert (np.abs(got[4:6]) <= 1e-36).all() and np.signbit(got[4:6]).all()
