"""Rotary positions of very many tokens on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402

pytestmark = pytest.mark.gpu


def test_more_tokens_than_a_launch_has_workgroups_in_a_row():
    """2^24 workgroups of 256 threads are 2^32 threads, one too many for a dimension of a grid."""
    T, D, half = (1 << 24) + 77, 16, 8
    x = torch.randn(T, 1, D, device="cuda", dtype=torch.float16)
    pos = torch.arange(T, device="cuda", dtype=torch.int64)
    f = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
    out = torch.full_like(x, float("nan"))
    w.rotary_axes(x, pos, f, out=out)
    for at in (0, (1 << 22) - 50, (1 << 23) - 50, (1 << 24) - 50, T - 100):
        rows = slice(at, at + 100)
        a = pos[rows, None].double() * f.double()
        c, s = a.cos(), a.sin()
        p, q = x[rows, 0, :half].double(), x[rows, 0, half:].double()
        want = torch.cat((p * c - q * s, q * c + p * s), -1)
        # half a step of fp16, and 8 steps of fp32 on |p| + |q| for the turn
        both = (p.abs() + q.abs()).repeat(1, 2)
        bound = 2.0 ** -25 + 2.0 ** -11 * want.abs() * 1.001 + 8 * 2.0 ** -24 * both
        assert bool(((out[rows, 0].double() - want).abs() <= bound).all())
    assert not bool(out.isnan().any())
