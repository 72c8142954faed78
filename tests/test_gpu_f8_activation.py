"""The gated product's activation on the GPU to fp32: the scale of a block with one value is that value / 448."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests import f8_util as f  # noqa: E402
from tests.f8_activation import U, activation  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m", [8, 60, 4000])
def test_to_fp32(m, kind):
    """g is the token's first scale, up or down, and u = 1 from the second block: all exact."""
    rng = np.random.default_rng(m)
    low = 80 if kind == "silu" else 9                      # beyond, scales are no normal fp32 numbers
    size = np.concatenate([np.exp(rng.uniform(-9, np.log(low), m // 2)), rng.uniform(0, low, m - m // 2)]).astype(np.float32)
    x = np.zeros((m, 256), np.float32)
    x[:, 0] = x[:, 128] = 1
    gate, up = np.zeros((256, 256), np.float32), np.zeros((256, 256), np.float32)
    gate[3, 0], gate[200, 0] = 1, -1                       # one value in each of two blocks of columns
    up[3, 128], up[200, 128] = 1, 1

    def f8(v):
        return torch.from_numpy(f.encode(v)).cuda().view(torch.float8_e4m3fn)

    ones = torch.ones(2, 2, device="cuda")
    sx = torch.from_numpy(np.stack([size, np.ones(m, np.float32)])).cuda()
    q, s = w.f8_gemm_gated(f8(x), sx, f8(gate), ones, f8(up), ones, kind)
    s, q = s.cpu().numpy().astype(np.float64), q.view(torch.uint8).cpu().numpy()
    for block, column, sign in ((0, 3, 1), (1, 200, -1)):
        want, bound = activation(sign * size.astype(np.float64), kind)
        # the scale's own rounding, and the smallest normal one
        assert (np.abs(s[block] * 448 - np.abs(want)) <= bound + 1.001 * U * np.abs(want) + 448 * 2.0 ** -126).all()
        seen = s[block] > 0
        assert (q[seen, column] == (0x7E if sign > 0 else 0xFE)).all()
        assert seen.sum() > m * 0.9
