"""Which kernels the 8-bit floating point products run with: every launch's part of the output, the
workspaces, and that the sizes tested on the GPU reach every kernel."""
import ctypes
import os
import random
import subprocess

import pytest

from tests.f8_paths import GATED, PRODUCTS

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "native", "f8_plan_shim.cpp")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FEW, TILE, LARGE = 0, 1, 2
TILES = [(64, 64), (64, 128), (96, 128), (128, 64), (128, 128)]


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    so = str(tmp_path_factory.mktemp("shim") / "f8_plan_shim.so")
    subprocess.run([HIPCC, "--offload-host-only", "-x", "hip", "-O1", "-std=c++17", "-fPIC", "-shared", SRC, "-o", so],
                   check=True, capture_output=True)
    L = ctypes.CDLL(so)
    L.shim_workspace.restype = L.shim_workspace_any.restype = ctypes.c_int64
    L.shim_workspace.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    L.shim_workspace_any.argtypes = [ctypes.c_int64] * 2
    return L


def plan(shim, M, N, K, gated, quantize, num_cu=256):
    out = (ctypes.c_int64 * 32)()
    n = shim.shim_plan(M, N, K, gated, quantize, num_cu, out)
    return [tuple(out[8 * i:8 * i + 7]) for i in range(n)]


def check(shim, M, N, K, gated, quantize, num_cu):
    launches = plan(shim, M, N, K, gated, quantize, num_cu)
    what = f"{M} {N} {K} {gated} {quantize} {num_cu}: {launches}"
    assert len(launches) in (1, 2), what
    # the parts lie side by side and make the whole
    assert launches[0][3:5] == (0, 0), what
    if len(launches) == 1:
        assert launches[0][5:] == (M, N), what
    else:
        (_, _, _, _, _, m, n), (_, _, _, m0, n0, m2, n2) = launches
        assert (m0, n0, m + m2, n, n2) == (m, 0, M, N, N) or (m0, n0, m, m2, n + n2) == (0, n, M, M, N), what
        assert launches[0][0] == LARGE and (n0 % 128 == 0), what
    need = shim.shim_workspace(M, N, K, gated, quantize)
    nb = -(-N // 128)
    for kind, shape, splits, _, _, m, n in launches:
        assert m > 0 and n > 0, what
        if kind == FEW:
            assert m <= 64 and 1 <= splits <= -(-K // 128) and (splits == 1 or not gated), what
            if splits > 1 or quantize:                     # sums of 128 columns for each range, and the counters
                assert need >= nb * splits * m * 512 + nb * 8, what
        elif kind == TILE:
            bm, bn = TILES[shape]
            tiles = -(-m // bm) * -(-n // bn)
            assert tiles * splits * 256 < 1 << 32, what
            if splits > 1:                                 # every part's sums of every tile, and the counters
                assert len(launches) == 1 and M > 64 and splits <= -(-K // 128) and not (quantize and bn < 128), what
                assert need >= splits * tiles * bm * bn * 4 * (1 + gated) + tiles * 8, what
            if quantize and bn < 128:                      # two workgroups a scale: one tile of tokens only
                assert m <= bm and need >= nb * m * 512 + nb * 8, what
        else:
            assert M > 64, what
    return launches


def test_parts_and_workspaces(shim):
    rng = random.Random(5)
    for num_cu in (256, 80, 304):
        for i in range(6000):
            top = rng.choice([70, 600, 5000, 60000, 1 << 25])
            M = rng.randint(1, top)
            N = rng.randint(1, rng.choice([300, 5000, 40000, 1 << 27 if M <= 4096 else 40000]))
            K = 16 * rng.randint(1, rng.choice([20, 400, 1 << 18]))
            gated = rng.randint(0, 1)
            check(shim, M, N, K, gated, gated and rng.randint(0, 1), num_cu)


def test_ends_of_the_ranges(shim):
    for M in (1, 32, 33, 64, 65, 1 << 25):
        for N in (1, 512, 513, 1024, 1025, 8128, 8129, 1 << 27):
            for K in (16, 8064, 8080, 1 << 22):
                for gated, quantize in ((0, 0), (1, 0), (1, 1)):
                    check(shim, M, N, K, gated, quantize, 256)


def test_workspace_for_any_columns(shim):
    """linear's workspace does not know N: the most that any N needs."""
    for M in (1, 2, 16, 33, 64, 65, 128, 300, 5000, 16384, 16385):
        for K in (16, 8064, 8080, 14336, 1 << 20):
            most = max(shim.shim_workspace(M, N, K, 0, 0) for N in list(range(1, 3000)) + [8128, 8129, 10240, 1 << 20])
            assert shim.shim_workspace_any(M, K) >= most


def test_gpu_sizes_reach_every_kernel(shim):
    def reached(sizes, gated, quantize):
        seen = set()
        for M, N, K in sizes:
            launches = check(shim, M, N, K, gated, quantize, 256)
            if len(launches) == 2:
                seen.add("tokens" if launches[1][3] else "columns")
            for kind, shape, splits, *_ in launches:
                seen.add({FEW: ("few", splits), TILE: ("tile", shape), LARGE: "large"}[kind])
                if kind == TILE and splits > 1:
                    seen.add("parts")
            if launches[0][0] == LARGE and len(launches) == 1:
                seen.add("large alone")
        return seen

    every = {("few", 1), "parts", "large", "large alone", "tokens", "columns"}
    assert reached(PRODUCTS, 0, 0) >= every | {("few", 2), ("few", 4)} | {("tile", i) for i in range(5)}
    assert reached(GATED, 1, 0) >= every | {("tile", i) for i in range(5)}
    assert reached(GATED, 1, 1) >= every | {("tile", i) for i in (0, 1, 2, 4)}
