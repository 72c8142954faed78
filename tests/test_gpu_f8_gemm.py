"""f8_gemm, f8_gemm_gated and linear(Mode.F8) against their definitions in 64 bits."""
import numpy as np
import pytest

from tests import f8_util as f
from tests.parity_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_gpu():
    return require_gpu()


def f8(codes):
    import torch
    return dev(codes).view(torch.float8_e4m3fn)


def codes_of(t):
    import torch
    return host(t.view(torch.uint8))


def codes(rng, r, c, wide=False):
    """e4m3 codes as quantised rows have them, or of every size."""
    if wide:
        q = rng.integers(0, 256, size=(r, c), dtype=np.uint8)
        q[(q & 127) == 127] = 0
        return q
    return f.encode(np.clip(rng.normal(size=(r, c)) * 110, -448, 448).astype(np.float32))


def operands(rng, m, n, k, wide=False, sides=1):
    """x with scales, and `sides` weights with scales: outputs of the size of 1 to 10."""
    blocks, nb = -(-k // 128), -(-n // 128)
    unit = 1 / (110 * 110 * np.sqrt(k))
    xq, sx = codes(rng, m, k, wide), np.exp(rng.normal(size=(blocks, m)) * 0.5).astype(np.float32)
    sx[rng.random(sx.shape) < 0.05] = 0
    ws = []
    for _ in range(sides):
        ws += [codes(rng, n, k, wide), (np.exp(rng.normal(size=(nb, blocks)) * 0.5) * unit).astype(np.float32)]
    return xq, sx, *ws


def on_gpu(xq, sx, *ws):
    return [f8(xq), dev(sx)] + [f8(t) if i % 2 == 0 else dev(t) for i, t in enumerate(ws)]


SHAPES = [(1, 1, 16), (1, 128, 128), (3, 5, 48), (16, 16, 144), (1, 300, 1040), (5, 129, 2560), (17, 64, 400), (33, 129, 272),
          (64, 200, 512), (70, 200, 400), (129, 257, 512), (200, 96, 656), (257, 130, 128), (300, 520, 144)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
def test_product(torch_gpu, m, n, k, wide):
    import w4a8_int8_gemm_amd as w
    data = operands(np.random.default_rng(m * 3 + n * 5 + k), m, n, k, wide)
    y = host(w.f8_gemm(*on_gpu(*data))).astype(np.float64)
    want, bound = f.product(*data)
    assert (np.abs(y - want) <= f.fp16_bound(want, bound)).all()


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated(torch_gpu, m, n, k, kind):
    import w4a8_int8_gemm_amd as w
    data = operands(np.random.default_rng(m + n + k), m, n, k, sides=2)
    g = on_gpu(*data)
    v, dv = f.gated(*data, kind)
    y = host(w.f8_gemm_gated(*g, kind, quantize=False)).astype(np.float64)
    assert (np.abs(y - v) <= f.fp16_bound(v, dv)).all()
    q, s = w.f8_gemm_gated(*g, kind)
    f.check_codes_f8(codes_of(q), host(s), v, dv, f"{m} {n} {k}")


def test_same_bits_every_call(torch_gpu):
    import torch
    import w4a8_int8_gemm_amd as w
    for m, n, k in ((1, 1000, 4096), (40, 700, 2048), (300, 900, 1024), (1025, 1100, 640)):
        g = on_gpu(*operands(np.random.default_rng(m), m, n, k, sides=2))
        first = w.f8_gemm(*g[:4]), *w.f8_gemm_gated(*g)
        for _ in range(3):
            again = w.f8_gemm(*g[:4]), *w.f8_gemm_gated(*g)
            for a, b in zip(first, again):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_scales_and_codes_that_are_no_numbers(torch_gpu):
    """A NaN scale reaches its token (or its 128 columns), a NaN code its row or column, and nothing else."""
    import w4a8_int8_gemm_amd as w
    for m, n, k in ((5, 300, 400), (70, 300, 400), (300, 300, 400)):
        xq, sx, wq, sw = operands(np.random.default_rng(m), m, n, k)
        clean = host(w.f8_gemm(*on_gpu(xq, sx, wq, sw)))
        bad = np.zeros((m, n), bool)
        sx2, sw2, xq2, wq2 = sx.copy(), sw.copy(), xq.copy(), wq.copy()
        sx2[1, 2] = np.nan
        bad[2] = True
        sw2[2, 3] = np.nan
        bad[:, 256:] = True
        xq2[0, 399] = 0x7F
        bad[0] = True
        wq2[7, 0] = 0xFF
        bad[:, 7] = True
        y = host(w.f8_gemm(*on_gpu(xq2, sx2, wq2, sw2)))
        assert np.isnan(y[bad]).all()
        np.testing.assert_array_equal(y[~bad], clean[~bad])
        # the gated product in 8 bits: the NaN takes its token's block, or for a weight's all tokens'
        g = on_gpu(xq2, sx2, wq, sw, wq2, sw)
        q, s = w.f8_gemm_gated(*g)
        s, c = host(s), codes_of(q)
        where = np.zeros(s.shape, bool)
        where[:, [0, 2]] = True
        where[0] = True
        assert (np.isnan(s) == where).all() and (c[2] == 0).all() and (c[:, :128] == 0).all()


@pytest.mark.parametrize("m,n,k", [(1, 77, 128), (3, 130, 272), (34, 133, 144), (65, 300, 256), (300, 261, 512)])
def test_outputs_end_where_they_end(torch_gpu, m, n, k):
    import torch
    import w4a8_int8_gemm_amd as w
    g = on_gpu(*operands(np.random.default_rng(m), m, n, k, sides=2))
    nb = -(-n // 128)
    y = torch.full((m * n + 4096,), 3.0, dtype=torch.float16, device="cuda")
    w.f8_gemm(*g[:4], out=y[: m * n].view(m, n))
    assert (y[m * n:] == 3).all()
    y.fill_(3)
    w.f8_gemm_gated(*g, quantize=False, out=y[: m * n].view(m, n))
    assert (y[m * n:] == 3).all()
    q = torch.full((m * n + 4096,), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((nb * m + 256,), 7.0, device="cuda")
    w.f8_gemm_gated(*g, out=q[: m * n].view(torch.float8_e4m3fn).view(m, n), scale=s[: nb * m].view(nb, m))
    assert (q[m * n:] == 77).all() and (s[nb * m:] == 7).all()


@pytest.mark.parametrize("m", [1, 6, 200])
def test_linear(torch_gpu, m):
    """linear(Mode.F8) is quantize_act_f8 and f8_gemm; without a workspace of the caller's too."""
    import torch
    import w4a8_int8_gemm_amd as w
    rng = np.random.default_rng(m)
    n, k = 330, 784
    x = rng.normal(size=(m, k)).astype(np.float16)
    wq, ws = w.quantize_weight_f8(dev((rng.normal(size=(n, k)) * 0.02).astype(np.float16)))
    y = w.linear(w.Mode.F8, dev(x), wq, ws)
    assert torch.equal(y, w.f8_gemm(*w.quantize_act_f8(dev(x)), wq, ws))
    assert torch.equal(y, w.linear_noalloc(w.Mode.F8, dev(x), wq, ws))
    xq, xs = f.rule(x, 1)
    want, bound = f.product(xq, np.ascontiguousarray(xs.T), codes_of(wq), host(ws))
    assert (np.abs(host(y) - want) <= f.fp16_bound(want, bound)).all()


def test_empty(torch_gpu):
    import torch
    import w4a8_int8_gemm_amd as w

    def e(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)

    def z(*shape):
        return torch.zeros(shape, device="cuda")

    assert w.f8_gemm(e(0, 128), z(1, 0), e(5, 128), z(1, 1)).shape == (0, 5)
    assert w.f8_gemm(e(3, 128), z(1, 3), e(0, 128), z(0, 1)).shape == (3, 0)
    q, s = w.f8_gemm_gated(e(3, 128), z(1, 3), e(0, 128), z(0, 1), e(0, 128), z(0, 1))
    assert q.shape == (3, 0) and s.shape == (0, 3)
    assert w.linear(w.Mode.F8, torch.zeros(0, 128, dtype=torch.float16, device="cuda"), e(5, 128), z(1, 1)).shape == (0, 5)


def test_another_stream_and_a_graph(torch_gpu):
    """Captured once, replayed with other inputs, eager work between the replays."""
    import torch
    import w4a8_int8_gemm_amd as w
    for m, n, k in ((1, 512, 1024), (40, 700, 2048), (300, 640, 1152)):
        sets = [on_gpu(*operands(np.random.default_rng(m + i), m, n, k, sides=2)) for i in range(3)]
        down = on_gpu(*operands(np.random.default_rng(9), m, k, 16 * (n // 16)))[2:]
        n16 = 16 * (n // 16)

        def both(g):
            q, s = w.f8_gemm_gated(*g)
            y = w.f8_gemm(*g[:4])
            return q, s, y, w.f8_gemm(q[:, :n16].contiguous(), s, *down)

        want = [both(g) for g in sets]
        static = [t.clone() for t in sets[0]]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both(static)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = both(static)
        for i in (1, 2, 0, 1):
            for a, b in zip(static, sets[i]):
                a.copy_(b)
            graph.replay()
            both(sets[(i + 1) % 3])
            torch.cuda.synchronize()
            for a, b in zip(out, want[i]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
