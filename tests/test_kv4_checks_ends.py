"""Arguments of the attention block at the ends of their ranges (no GPU needed)."""
import pytest

pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.test_kv4_checks import MIS, S, attention  # noqa: E402


@pytest.mark.parametrize("scale", [2.0 ** 127 * 1.01, 3e38, 3.4e38])
def test_scales_whose_exponent_leaves_fp32(scale):
    """scale * log2(e) has to be finite."""
    assert attention(scale=scale) == S.ERR_INVALID_ARG
    assert attention(scale=2.0 ** 127, q=MIS) == S.ERR_ALIGNMENT      # taken; what is refused comes later
    assert w.lib().w4a8_last_error()
