"""The 8-bit floating point products at the ends of their tiles and ranges: tiles of the large kernel without a
second half, one block of K in its stream of stages, and the largest K."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests import f8_util as f  # noqa: E402
from tests.test_gpu_f8_paths import F8, check_codes, check_half, gated, operands, product  # noqa: E402

pytestmark = pytest.mark.gpu


# plain: the large kernel alone; with 128 and more stages of K and few, whole blocks of K and not, N 1 to 128
# past a multiple of 256
@pytest.mark.parametrize("m,n,k", [(20000, 1290, 272), (1500, 16394, 272), (20000, 1290, 384), (20000, 1408, 400), (8200, 1281, 2064)])
def test_tiles_without_a_second_half(m, n, k):
    data = operands(m, n, k, m + n + k)
    check_half(w.f8_gemm(*data), *product(*data))
    # scales that are no numbers in the last block reach its columns and no others
    data[3][-1, -1] = float("nan")
    y = w.f8_gemm(*data)
    last = (n - 1) // 128 * 128
    assert y[:, last:].isnan().all() and not y[:, :last].isnan().any()


def ends(total, block):
    at = sorted({0, 1, total // block // 2, (total - 1) // block - 1, (total - 1) // block})
    return torch.cat([torch.arange(b * block, min(total, (b + 1) * block), device="cuda") for b in at])


@pytest.mark.parametrize("k", [16, 128])
@pytest.mark.parametrize("form", ["e4m3", "fp16"])
def test_one_block_of_k_in_large_tiles(form, k):
    """So many tiles that only the large kernel numbers them, each of one stage: every stage of the stream is a
    tile's first and last.  64 and 128 GiB of output, of which the first and last tiles and some between."""
    m, n = (1 << 18) + 5, (1 << 18) + 64
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 * 2 ** 30:
        pytest.skip("200 GiB of free memory")
    g = torch.Generator(device="cuda").manual_seed(k)

    def codes(r):
        return (torch.randn(r, k, device="cuda", generator=g) * 110).clamp(-448, 448).to(F8)

    xq, wq, up = codes(m), codes(n), codes(n)
    sx = torch.rand(1, m, device="cuda", generator=g) + 0.5
    sw = (torch.rand(-(-n // 128), 1, device="cuda", generator=g) + 0.5) / (110 * 110 * k ** 0.5)
    rows, cols = ends(m, 128), ends(n, 128)

    def pick(t, at):
        return t.view(torch.uint8)[at].view(F8)

    blocks = torch.unique(cols // 128)
    some = pick(xq, rows), sx[:, rows].contiguous(), pick(wq, cols), sw[blocks], pick(up, cols), sw[blocks]
    if form == "fp16":
        y = w.f8_gemm(xq, sx, wq, sw)
        got = y[rows][:, cols]
        del y
        check_half(got, *product(*some[:4]))
    else:
        q, s = w.f8_gemm_gated(xq, sx, wq, sw, up, sw)
        got, s = q.view(torch.uint8)[rows][:, cols].view(F8), s[blocks][:, rows]
        del q
        check_codes(got, s, *gated(*some, "silu"))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n", [(1, 40), (64, 130), (130, 70)])
def test_the_largest_k(m, n):
    data = operands(m, n, 2 ** 22, m)
    check_half(w.f8_gemm(*data), *product(*data))


def test_quantizers_at_the_largest_k():
    rng = np.random.default_rng(1)
    x = (rng.normal(size=(1, 2 ** 22)) * np.exp(rng.uniform(-8, 6, size=2 ** 22))).astype(np.float16)
    for quantize, rows in ((w.quantize_act_f8, 1), (w.quantize_weight_f8, 128)):
        q, s = quantize(torch.from_numpy(x).cuda())
        want, ws = f.rule(x, rows)
        np.testing.assert_array_equal(s.cpu().numpy(), ws.T if rows == 1 else ws)
        np.testing.assert_array_equal(q.view(torch.uint8).cpu().numpy(), want)
