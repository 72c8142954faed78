"""Attention over the 4-bit cache where its arguments and its cache are at their ends, against the
definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.test_gpu_kv4_attention import Case, dev  # noqa: E402

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("kv,m", [([0, 4, 1], [5, 9, 2]), ([0, 4, 1], [40, 70, 33]), ([3, 100, 1], [200, 150, 300])])
@pytest.mark.parametrize("window", [TOP, TOP - 1, 2 ** 30])
def test_the_largest_windows(kv, m, window):
    """More queries than keys, so that the first key of a window lies below -2^31."""
    Case(kv, m, 4, 2, 128, 128, 16, seed=21).check(window=window)
