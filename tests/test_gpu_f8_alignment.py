"""What a block's sum of the 8-bit products keeps, to fp32: the gated product with gates of 64 (silu gives 64
again), of whose output in e4m3 a block with one value has the scale 64 P / 448."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests import f8_util as f  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def sums(x, weights, m):
    """P of the first 128 of K from codes' values x [128] and weights [cases, 128], each case in a block of
    columns of its own; m tokens, all alike."""
    n = 128 * len(weights)
    xs, gate, up = np.zeros((m, 256)), np.zeros((n, 256)), np.zeros((n, 256))
    xs[:, :128], xs[:, 128] = x, 8
    gate[::128, 128] = 8
    up[::128, :128] = weights

    def f8(v):
        q = f.encode(v.astype(np.float32))
        assert (f.decode(q) == v).all()
        return torch.from_numpy(q).cuda().view(torch.float8_e4m3fn)

    sx, sw = torch.ones(2, m, device="cuda"), torch.ones(len(weights), 2, device="cuda")
    _, s = w.f8_gemm_gated(f8(xs), sx, f8(gate), sw, f8(up), sw)
    s = s.cpu().numpy().astype(np.float64) * 7             # 448 / 64
    assert (s == s[:, :1]).all()
    return s[:, 0]


@pytest.mark.parametrize("m", [3, 40, 300])
def test_sums_within_13_bits_are_exact(m):
    """Neighbours within 2^12 of each other in whole units of the last: nothing is dropped."""
    rng = np.random.default_rng(m)
    weights = np.zeros((64, 128))
    for case in weights:                                   # powers of two from 1 to 256, and ones
        case[:] = 2.0 ** rng.integers(0, 9, 128)
    x = np.where(np.arange(128) % 8 == 0, 8.0, 1.0)
    got, want = sums(x, weights, m), weights @ x
    assert (np.abs(got - want) <= 2 * U * want).all()      # the scale's quotient, and 7 s


@pytest.mark.parametrize("m", [3, 40, 300])
def test_what_lies_below_is_dropped_and_no_more(m):
    """Every eight: one product of 2^e and seven of up to 15/8 2^(e - 14), just below 2^-13 of it."""
    rng = np.random.default_rng(m)
    weights = np.zeros((64, 128))
    x = np.full(128, 2.0 ** -6)
    x[::8] = 1
    for i, case in enumerate(weights):
        case[:] = (1 + rng.integers(0, 8, 128) / 8) * 2.0 ** -6 if i else 15 / 8 * 2.0 ** -6
        case[::8] = 4
    got, want = sums(x, weights, m), weights @ x
    dropped = 7 * 16 * 2.0 ** (2 - 13.0)
    assert ((want - got >= -2 * U * want) & (want - got <= dropped + 2 * U * want)).all()
    assert dropped <= 8.6e-4 * want.min()
