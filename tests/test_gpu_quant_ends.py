"""Quantizing very many rows on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,K", [(0, 8), (64, 64)])
def test_more_rows_than_one_launch_holds(group, K):
    """Four rows a workgroup of 256 threads: 2^26 rows are 2^32 threads.  Rows at the ends and at the borders
    equal those of a call of their own."""
    M = (1 << 26) + 77
    x = torch.empty((M, K), device="cuda", dtype=torch.float16)
    x.normal_()
    q = torch.zeros((M, K), device="cuda", dtype=torch.int8)
    s = torch.full((M,) if group == 0 else (M, K // group), float("nan"), device="cuda")
    w.quantize_act(x, group, out=q, scale=s)
    for at in (0, (1 << 24) - 50, (1 << 25) - 50, (1 << 26) - 50, M - 100):
        rows = slice(at, at + 100)
        a, b = w.quantize_act(x[rows].clone(), group)
        assert torch.equal(q[rows], a) and torch.equal(s[rows], b)
    assert not bool(s.isnan().any())
