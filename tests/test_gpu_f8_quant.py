"""quantize_act_f8, quantize_weight_f8 and rmsnorm_quant against their definitions in 64 bits."""
import numpy as np
import pytest

from tests import f8_util as f
from tests.parity_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_gpu():
    return require_gpu()


def codes_of(t):
    import torch
    return host(t.view(torch.uint8))


def rows(rng, m, k, spread=True):
    x = rng.normal(size=(m, k)).astype(np.float32)
    if spread:
        x *= np.exp(rng.uniform(-9, 6, size=(m, 1)))
        x[:, ::37] *= 30
    return np.clip(x, -60000, 60000).astype(np.float16)


SHAPES = [(1, 8), (1, 16), (3, 128), (5, 136), (2, 504), (7, 512), (33, 520), (4, 1032), (130, 2560), (1, 4096),
          (2, 16640)]


@pytest.mark.parametrize("m,k", SHAPES)
def test_activations(torch_gpu, m, k):
    import w4a8_int8_gemm_amd as w
    x = rows(np.random.default_rng(m * 7 + k), m, k)
    x[0, : min(k, 128)] = 0                                       # a block of zeros
    x[-1, -8:] = np.float16(2.0 ** -24)                           # the smallest values
    q, s = w.quantize_act_f8(dev(x))
    want, ws = f.rule(x, 1)
    np.testing.assert_array_equal(host(s), ws.T)
    np.testing.assert_array_equal(codes_of(q), want)


@pytest.mark.parametrize("n,k", [(1, 8), (3, 136), (128, 128), (129, 264), (300, 1000), (4, 4104), (1000, 48)])
def test_weights(torch_gpu, n, k):
    import w4a8_int8_gemm_amd as w
    x = rows(np.random.default_rng(n + k), n, k)
    x[:, -5:] = 0
    q, s = w.quantize_weight_f8(dev(x))
    want, ws = f.rule(x, 128)
    np.testing.assert_array_equal(host(s), ws)
    np.testing.assert_array_equal(codes_of(q), want)


def test_every_value_of_a_block_scale(torch_gpu):
    """All fp16 values up to a few block maxima: ties between codes and subnormal codes among them."""
    import w4a8_int8_gemm_amd as w
    bits = np.arange(0x7C00, dtype=np.uint16)
    for top in (0x5F00, 0x3C00, 0x0400, 0x0011, 0x7BFF, 0x49A3):
        v = bits[: top + 1].view(np.float16)
        v = np.concatenate([v, np.zeros(-len(v) % 127, np.float16)]).reshape(-1, 127)
        x = np.concatenate([np.full((len(v), 1), np.uint16(top).view(np.float16)), v * np.float16(-1)], 1)
        q, s = w.quantize_act_f8(dev(x))
        want, ws = f.rule(x, 1)
        np.testing.assert_array_equal(host(s), ws.T)
        np.testing.assert_array_equal(codes_of(q), want)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_values_that_are_not_finite_stay_in_their_block(torch_gpu, bad):
    import w4a8_int8_gemm_amd as w
    x = rows(np.random.default_rng(3), 6, 400)
    y = x.copy()
    y[2, 140] = bad
    q0, s0 = w.quantize_act_f8(dev(x))
    q1, s1 = w.quantize_act_f8(dev(y))
    a, b, sa, sb = codes_of(q0), codes_of(q1), host(s0), host(s1)
    assert np.isnan(sb[1, 2]) and (b[2, 128:256] == 0).all()
    sa[1, 2] = sb[1, 2] = 0
    b[2, 128:256] = a[2, 128:256]
    np.testing.assert_array_equal(sa, sb)
    np.testing.assert_array_equal(a, b)
    q2, s2 = w.quantize_weight_f8(dev(y))
    assert np.isnan(host(s2)[0, 1]) and np.isfinite(host(s2)[0, [0, 2, 3]]).all()
    assert (codes_of(q2)[:, 128:256] == 0).all()


def check_norm(w, mode, gs, x, gain, eps, residual, got):
    codes, scale = got[:2]
    v, dv, h = f.norm(x, gain, eps, residual)
    m, k = x.shape
    if residual is not None:
        with np.errstate(over="ignore"):
            want = h.astype(np.float32).astype(np.float16)        # the sum in fp32, then one rounding
        np.testing.assert_array_equal(host(got[2]), want)
    if mode == w.Mode.F8:
        assert scale.shape == (-(-k // 128), m)
        f.check_codes_f8(codes_of(codes), host(scale), v, dv)
        return
    group = gs or k
    s = host(scale).reshape(m, -1).astype(np.float64)
    q = host(codes).astype(np.float64)
    vv, dd = v.reshape(m, -1, group), dv.reshape(m, -1, group)
    top = np.abs(vv).max(-1)
    ds = dd.max(-1) / 127 + 2 * f.U * top / 127
    assert (np.abs(s - top / 127) <= ds * 1.001 + 2.0 ** -126).all()
    assert (np.abs(q) <= 127).all()
    off = np.abs(q.reshape(vv.shape) * s[..., None] - vv)
    assert (off <= s[..., None] * (0.5 + 2.0 ** -16) + dd * 1.001 + 128 * ds[..., None] * 2.0 ** -8).all()


MODES = [("F8", 0), ("W8A8_PC", 0), ("W4A8", 0), ("W8A8_PG", 64), ("W8A8_PG", 128)]


@pytest.mark.parametrize("mode,gs", MODES)
@pytest.mark.parametrize("m,k", [(1, 128), (3, 384), (1, 4096), (5, 2560), (130, 1152), (2, 8192), (9, 5120), (4, 14336), (2, 16640),
                                 (3, 33280)])
@pytest.mark.parametrize("add", [False, True])
def test_norm(torch_gpu, mode, gs, m, k, add):
    import w4a8_int8_gemm_amd as w
    mode = w.Mode[mode]
    rng = np.random.default_rng(m + k + gs)
    x, gain = rows(rng, m, k), (1 + 0.3 * rng.normal(size=k)).astype(np.float16)
    r = rows(rng, m, k, False) if add else None
    eps = 1e-5
    got = w.rmsnorm_quant(mode, dev(x), dev(gain), eps, residual=None if r is None else dev(r), group_size=gs)
    assert len(got) == (3 if add else 2)
    check_norm(w, mode, gs, x, gain, eps, r, got)


@pytest.mark.parametrize("m,k", [(1, 8), (2, 24), (1, 72), (6, 136), (3, 1000), (5, 2056), (2, 4104), (3, 8200), (2, 17000)])
@pytest.mark.parametrize("mode", ["F8", "W8A8_PC"])
def test_norm_of_odd_widths(torch_gpu, mode, m, k):
    import w4a8_int8_gemm_amd as w
    mode = w.Mode[mode]
    rng = np.random.default_rng(m + k)
    x, gain, r = rows(rng, m, k), rng.normal(size=k).astype(np.float16), rows(rng, m, k)
    check_norm(w, mode, 0, x, gain, 0.0, None, w.rmsnorm_quant(mode, dev(x), dev(gain), 0.0))
    check_norm(w, mode, 0, x, gain, 0.1, r, w.rmsnorm_quant(mode, dev(x), dev(gain), 0.1, residual=dev(r)))


@pytest.mark.parametrize("mode,gs", MODES)
def test_norm_rows_of_zeros_and_of_no_numbers(torch_gpu, mode, gs):
    import w4a8_int8_gemm_amd as w
    mode = w.Mode[mode]
    k = 1280
    rng = np.random.default_rng(1)
    x = rows(rng, 9, k, False)
    gain = np.ones(k, np.float16)
    gain[256:384] = 0                                              # a block whose gains are zero
    x[1] = 0
    clean = w.rmsnorm_quant(mode, dev(x), dev(gain), 0.0, group_size=gs)
    y = x.copy()
    y[3, 700], y[5, 2], y[7, 1279] = np.nan, np.inf, -np.inf
    got = w.rmsnorm_quant(mode, dev(y), dev(gain), 0.0, group_size=gs)

    def by_row(t):
        s = host(t)
        return s.T if mode == w.Mode.F8 else s.reshape(9, -1)

    a, b = by_row(clean[1]), by_row(got[1])
    ca, cb = (host(c[0].view(torch_gpu.uint8)) for c in (clean, got))
    assert (a[1] == 0).all() and (ca[1] == 0).all()
    if mode == w.Mode.F8:
        assert (a[:, 2] == 0).all()
    for i in range(9):
        if i in (3, 5, 7):
            assert np.isnan(b[i]).all() and (cb[i] == 0).all()
        else:
            np.testing.assert_array_equal(a[i], b[i])
            np.testing.assert_array_equal(ca[i], cb[i])


def test_norm_of_sums_beyond_fp16(torch_gpu):
    """h is held in fp32: its norm is right where fp16(h) is infinite or has lost the addend."""
    import w4a8_int8_gemm_amd as w
    rng = np.random.default_rng(2)
    x, r = rows(rng, 4, 512, False), rows(rng, 4, 512, False)
    x[0], r[0] = 60000, 50000
    x[1] *= np.float16(2.0 ** -10)
    r[1] *= np.float16(1000)
    gain = np.ones(512, np.float16)
    for mode in (w.Mode.F8, w.Mode.W8A8_PC):
        check_norm(w, mode, 0, x, gain, 1e-6, r, w.rmsnorm_quant(mode, dev(x), dev(gain), 1e-6, residual=dev(r)))


@pytest.mark.parametrize("k", [264, 4096, 9216, 20000])
def test_norm_in_place(torch_gpu, k):
    """The residual's stream (or x) may be the sum's place."""
    import w4a8_int8_gemm_amd as w
    rng = np.random.default_rng(k)
    x, r, gain = rows(rng, 37, k, False), rows(rng, 37, k, False), rng.normal(size=k).astype(np.float16)
    for mode in (w.Mode.F8, w.Mode.W8A8_PC):
        q, s, h = w.rmsnorm_quant(mode, dev(x), dev(gain), residual=dev(r))
        for place in (0, 1):
            xd, rd = dev(x), dev(r)
            got = w.rmsnorm_quant(mode, xd, dev(gain), residual=rd, residual_out=(xd, rd)[place])
            assert got[2].data_ptr() == (xd, rd)[place].data_ptr()
            for a, b in zip((q, s, h), got):
                np.testing.assert_array_equal(host(a.view(torch_gpu.uint8)), host(b.view(torch_gpu.uint8)))


def test_outputs_end_where_they_end(torch_gpu):
    """Nothing is written behind the rows, of codes, scales and sums."""
    import torch
    import w4a8_int8_gemm_amd as w
    for m, k in ((1, 264), (5, 136), (3, 4104), (2, 17000)):
        x = dev(rows(np.random.default_rng(m), m, k))
        blocks = -(-k // 128)
        for act in (True, False):
            codes = torch.full((m * k + 512,), 77, dtype=torch.uint8, device="cuda")
            scale = torch.full((blocks * m + 64,), 7.0, device="cuda")
            total = torch.full((m * k + 64,), 3.0, dtype=torch.float16, device="cuda")
            q = codes[: m * k].view(torch.float8_e4m3fn).view(m, k)
            s = scale[: blocks * m].view(blocks, m)
            if act:
                w.quantize_act_f8(x, out=q, scale=s)
            else:
                w.rmsnorm_quant(w.Mode.F8, x, torch.ones(k, dtype=torch.float16, device="cuda"), residual=x, out=q,
                                scale=s, residual_out=total[: m * k].view(m, k))
            assert (codes[m * k:] == 77).all() and (scale[blocks * m:] == 7).all() and (total[m * k:] == 3).all()


def test_empty_and_other_streams(torch_gpu):
    import torch
    import w4a8_int8_gemm_amd as w
    q, s = w.quantize_act_f8(torch.empty(0, 256, dtype=torch.float16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (2, 0)
    got = w.rmsnorm_quant(w.Mode.W8A8_PC, torch.empty(0, 256, dtype=torch.float16, device="cuda"),
                          torch.empty(256, dtype=torch.float16, device="cuda"))
    assert got[0].shape == (0, 256) and got[1].shape == (0,)
    x = dev(rows(np.random.default_rng(1), 600, 4096))
    gain = torch.ones(4096, dtype=torch.float16, device="cuda")
    want = w.rmsnorm_quant(w.Mode.F8, x, gain)
    side = torch.cuda.Stream()
    y = torch.empty_like(x)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y.copy_(x)
        got = w.rmsnorm_quant(w.Mode.F8, y, gain)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_norm_of_more_rows_than_a_launch_has(torch_gpu):
    """2^21 rows a launch; the rows behind are those of the next."""
    import torch
    import w4a8_int8_gemm_amd as w
    m, k = (1 << 21) + 3, 16
    x = torch.zeros(m, k, dtype=torch.float16, device="cuda")
    x[-5:] = torch.arange(1, 81, device="cuda").view(5, 16).half()
    gain = torch.ones(k, dtype=torch.float16, device="cuda")
    for mode in (w.Mode.F8, w.Mode.W8A8_PC):
        q, s = w.rmsnorm_quant(mode, x, gain)
        a, b = w.rmsnorm_quant(mode, x[-5:].contiguous(), gain)
        assert torch.equal(q[-5:].view(torch.uint8), a.view(torch.uint8))
        assert torch.equal(s.flatten()[-5:], b.flatten())
        assert not q[:-5].view(torch.uint8).any() and not s.flatten()[:-5].any()


def test_activations_of_more_runs_than_a_launch_has(torch_gpu):
    """Rows of two runs of 512 values, one more than a launch numbers: each run's wavefront takes both."""
    import torch
    import w4a8_int8_gemm_amd as w
    m, k = (1 << 24) + 3, 520
    x = torch.zeros(m, k, dtype=torch.float16, device="cuda")
    x[-5:] = torch.randn(5, k, device="cuda").half()
    q, s = w.quantize_act_f8(x)
    a, b = w.quantize_act_f8(x[-5:].contiguous())
    assert torch.equal(q[-5:].view(torch.uint8), a.view(torch.uint8)) and torch.equal(s[:, -5:], b)
    assert not q[:-5].view(torch.uint8).any() and not s[:, :-5].any()
