"""rmsnorm_quant of rows so long that the order and the width of the squares' sum show."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# Of a value, relative: the sum's eight roundings in a row, its own to fp32, the mean's and the addition of eps,
# halved by the root; the root, the quotient and two products; h's rounding, in the sum and in itself.
VALUE = ((8 + 1 + 1 + 1) / 2 + 4 + 2) * U


def rows(k, add):
    rng = np.random.default_rng(k)
    first = np.full(k, 0.5)
    first[:512] = 1000                                     # a sum that is large before the many small squares
    x = np.stack([np.full(k, 0.1), np.full(k, 1.3), rng.normal(size=k), first, rng.normal(size=k) * np.exp(rng.uniform(-8, 4, k))])
    return x.astype(np.float16), (rng.normal(size=x.shape) * 0.01).astype(np.float16) if add else None


@pytest.mark.parametrize("k", [16392, 17000, 65536, 2 ** 20, 2 ** 22])
@pytest.mark.parametrize("mode", ["F8", "W8A8_PC"])
@pytest.mark.parametrize("add", [False, True])
def test_scales(k, mode, add):
    """The scales are the largest values / 448 or / 127: as near to those in 64 bits as the roundings allow."""
    mode = w.Mode[mode]
    x, r = rows(k, add)
    gain = (1 + 0.1 * np.random.default_rng(3).normal(size=k)).astype(np.float16)
    dev = [None if t is None else torch.from_numpy(t).cuda() for t in (x, gain, r)]
    q, s = w.rmsnorm_quant(mode, dev[0], dev[1], 1e-5, residual=dev[2])[:2]
    h = dev[0].double() + (dev[2].double() if add else 0)
    v = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * dev[1].double()
    if mode == w.Mode.F8:
        top = torch.nn.functional.pad(v.abs(), (0, -k % 128)).view(len(x), -1, 128).amax(2) / 448
        s, block = s.double().t(), 128
    else:
        top, s, block = v.abs().amax(1, keepdim=True) / 127, s.double()[:, None], k
    assert ((s - top).abs() <= 1.001 * (VALUE + U) * top).all()
    # the codes: half a step, of the value (or of the subnormals) or of the scale
    wide = s.repeat_interleave(block, 1)[:, :k]
    got = (q.double() if mode == w.Mode.F8 else q.to(torch.float64)) * wide
    half = torch.maximum(v.abs() * 2.0 ** -4, wide * 2.0 ** -10) if mode == w.Mode.F8 else wide / 2
    assert ((got - v).abs() <= 1.001 * half + (VALUE + U) * 1.1 * (v.abs() + 448 * wide * 2.0 ** -4)).all()
