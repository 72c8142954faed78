"""The 8-bit floating point quantizers at the end of their widths, before anything reaches a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402

P = ctypes.c_void_p
A, B, C = (P(4096 * i) for i in range(1, 4))


@pytest.mark.parametrize("k", [(1 << 22) + 8, 1 << 23, (1 << 31) - 512, (1 << 31) - 8, 1 << 31, 1 << 40])
@pytest.mark.parametrize("rows", [0, 1, 5])
@pytest.mark.parametrize("name", ["quantize_act_f8", "quantize_weight_f8"])
def test_wider_than_the_products_take(name, rows, k):
    """K is at most 2^22, as for the products and the norm (the header says so of all of them)."""
    L = w.lib()
    assert getattr(L, name)(A, rows, k, B, C, None) == int(w.Status.ERR_INVALID_ARG)
    assert str(k) in L.w4a8_last_error().decode()


@pytest.mark.parametrize("name", ["quantize_act_f8", "quantize_weight_f8"])
def test_the_widest(name):
    assert getattr(w.lib(), name)(None, 0, 1 << 22, None, None, None) == int(w.Status.OK)
