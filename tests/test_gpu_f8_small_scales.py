"""Codes of values so small that a residual in fp32 would underflow, bit for bit: the gated product's output
in e4m3, and the norm with an eps that makes its values as small."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests import f8_util as f  # noqa: E402

pytestmark = pytest.mark.gpu

# Largest values of a block (times a power of two) at which, with scales next to 2^-126, a quotient that is
# corrected by a residual below 2^-149 gives another code than the division for several of the values that
# lie nearest to the borders between codes.
TOPS = [14674450, 16516352, 14793506, 12849034, 16500265, 13719973, 16441130, 9215477]
EXPONENTS = [20, 96, 104, 110, 112, 116, 120, 124, 128, 132, 134, 136, 137, 138, 139]


def near_borders(top):
    """128 integers below 2^24, the largest first, then those nearest to the borders by its scale."""
    grid = f.decode(np.arange(127, dtype=np.uint8))
    s = float(np.float32(np.float32(top) / np.float32(448)))
    n = np.rint((grid[1:] + grid[:-1]) / 2 * s).astype(np.int64)
    return np.concatenate([[top], np.minimum(n, top), [0]])


def gated_operands(tokens, columns):
    """x [m, 384] and weights whose gates are 64 (silu gives 64 again, 1 + e^-64 being 1) and whose up values are
    `columns` (24-bit integers) times 2^-e of the token's e / 64: in the first block their lower 12 bits, in the
    second, with a scale 2^12 times as large, the upper ones, in the third the gates.  Every product and sum
    is exact: a code is a power of two, eight neighbours within 2^8 of each other."""
    m, n = len(tokens), len(columns)
    x = np.zeros((m, 384))
    for b in (0, 1):
        x[:, b * 128:b * 128 + 8], x[:, b * 128 + 8:b * 128 + 16] = 1, 16
    x[:, 256] = 8
    up, gate = np.zeros((n, 384)), np.zeros((n, 384))
    for b in (0, 1):
        part = (columns >> (12 * b)) & 4095
        for j in range(12):
            up[:, b * 128 + j] = ((part >> j) & 1) * 2.0 ** (j if j < 8 else j - 4)
    gate[:, 256] = 8
    e = np.asarray(tokens, np.float64)
    sx = np.stack([2.0 ** -(e + 6), 2.0 ** -(e - 6), np.ones(m)]).astype(np.float32)
    ones = np.ones((-(-n // 128), 3), np.float32)

    def f8(v):
        return torch.from_numpy(f.encode(v.astype(np.float32))).cuda().view(torch.float8_e4m3fn)

    xq, up, gate = f8(x), f8(up), f8(gate)
    dev = torch.from_numpy
    return xq, dev(sx).cuda(), gate, dev(ones).cuda(), up, dev(ones).cuda()


# the kernels for few tokens (its workgroups meet), for 64 tokens, tiles and large tiles
@pytest.mark.parametrize("m,blocks", [(3, 8), (15, 8), (40, 8), (50, 70), (74, 8), (300, 50), (2058, 60)])
def test_gated(m, blocks):
    tokens = [EXPONENTS[i % len(EXPONENTS)] for i in range(m - 3, -3, -1)]
    tops = [near_borders(t) for t in TOPS]
    columns = np.concatenate([tops[b % 8] for b in range(blocks)])
    data = gated_operands(tokens, columns)
    for kind in ("silu", "gelu_tanh"):
        q, s = w.f8_gemm_gated(*data, kind)
        q, s = q.view(torch.uint8).cpu().numpy(), s.cpu().numpy()
        for e in sorted(set(tokens)):
            v = np.ldexp(np.concatenate(tops).astype(np.float64), -e)[None]
            want, ws = f.rule(v, 1)
            assert (ws >= 2.0 ** -126).all()
            rows = np.flatnonzero(np.asarray(tokens) == e)
            want = np.concatenate([want[0, 128 * (b % 8):128 * (b % 8) + 128] for b in range(blocks)])
            assert (s[:, rows] == np.concatenate([ws[0]] * (blocks // 8 + 1))[:blocks, None]).all(), e
            assert (q[rows] == want).all(), e


@pytest.mark.parametrize("k", [128, 2048, 16640])
@pytest.mark.parametrize("mode,gs", [("F8", 0), ("W8A8_PC", 0), ("W8A8_PG", 64)])
def test_norm(k, mode, gs):
    """eps = 2^126 outweighs any row: v = h gain 2^-63 exactly, and every code is the division's."""
    rng = np.random.default_rng(k)
    m = 9
    h = (rng.integers(-2047, 2048, (m, k)) * 2.0 ** rng.integers(-24, -10, (m, 1))).astype(np.float16)
    gain = (rng.integers(0, 2048, k) * 2.0 ** -24).astype(np.float16)
    mode = w.Mode[mode]
    q, s = w.rmsnorm_quant(mode, torch.from_numpy(h).cuda(), torch.from_numpy(gain).cuda(), 2.0 ** 126, group_size=gs)
    v = h.astype(np.float64) * gain.astype(np.float64) * 2.0 ** -63
    if mode == w.Mode.F8:
        want, ws = f.rule(v, 1)
        np.testing.assert_array_equal(s.cpu().numpy().T, ws)
        np.testing.assert_array_equal(q.view(torch.uint8).cpu().numpy(), want)
        return
    b = v.reshape(m, -1, gs or k)
    ws = (np.abs(b).max(-1, keepdims=True) / 127).astype(np.float32)
    t = (b / ws).astype(np.float32).astype(np.float64)
    want = np.copysign(np.floor(np.abs(t) + 0.5), t).reshape(m, k)
    np.testing.assert_array_equal(s.cpu().numpy().reshape(m, -1), ws[..., 0])
    np.testing.assert_array_equal(q.cpu().numpy(), want)
