"""Rotary positions on the GPU against their definition in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.kv4_util import HALF_ROUND, HALF_TINY, U  # noqa: E402

pytestmark = pytest.mark.gpu


def axis_of(i, sections, interleaved):
    if interleaved:
        a = i % len(sections)
        return a if i // len(sections) < sections[a] else 0
    for a, n in enumerate(sections):
        if i < n:
            return a
        i -= n
    raise AssertionError


def reference(x, pos, freq, sections, interleaved):
    """x fp16 [T, h, d], pos [axes, T], freq fp32 -> (y, bound), fp64.

    The angle is reduced to a turn in fp64 and rounded to fp32 as a fraction (at most 2^-25 of a
    turn, 2 pi 2^-25 = 3.2 u); cosine and sine are off by at most 2 u more each, a product and an
    fma by u each: 8 u on |a| + |b|, then half a step of fp16."""
    y = x.astype(np.float64)
    b = HALF_TINY + HALF_ROUND * np.abs(y)
    half = len(freq)
    for i in range(half):
        ang = pos[axis_of(i, sections, interleaved)].astype(np.float64) * float(freq[i])
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        p, q = x[..., i].astype(np.float64), x[..., i + half].astype(np.float64)
        y[..., i], y[..., i + half] = p * c - q * s, q * c + p * s
        for at in (i, i + half):
            b[..., at] = HALF_TINY + HALF_ROUND * np.abs(y[..., at]) * 1.001 + 8 * U * (np.abs(p) + np.abs(q))
    return y, b


def freqs(half, theta=1e6):
    return (1.0 / theta ** (np.arange(half) / half)).astype(np.float32)


def inputs(T, heads, D, axes, seed, far=1 << 20):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, heads, D)).astype(np.float16)
    pos = r.integers(0, far, (axes, T), dtype=np.int64)
    return x, pos


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("T,heads,D,R,sections,interleaved", [
    (1, 40, 128, 128, (24, 20, 20), True),
    (1, 1, 64, 64, (32,), False),
    (2, 3, 64, 32, (8, 8), True),
    (5, 7, 256, 256, (128,), True),
    (17, 40, 128, 128, (24, 20, 20), False),
    (33, 5, 128, 64, (0, 16, 16), False),
    (33, 5, 128, 64, (32, 0, 0), True),
    (64, 9, 80, 16, (3, 3, 2), True),
    (129, 12, 256, 128, (22, 21, 21), True),
    (300, 1, 1024, 1024, (200, 156, 156), False),
    (1000, 2, 8 * 3, 16, (8,), False),
])
def test_matches_the_definition(T, heads, D, R, sections, interleaved):
    x, pos = inputs(T, heads, D, len(sections), seed=T + D)
    f = freqs(R // 2)
    y, b = reference(x, pos, f, sections, interleaved)
    out = w.rotary_axes(dev(x), dev(pos), dev(f), sections, interleaved)
    got = out.cpu().numpy().astype(np.float64)
    assert out.shape == x.shape and (np.abs(got - y) <= b).all(), float((np.abs(got - y) / b).max())


def test_far_negative_and_zero_positions():
    x, _ = inputs(6, 4, 128, 1, seed=1)
    pos = np.array([[0, -1, 1, 2 ** 31 - 1, -2 ** 31, 123456789]], np.int64)
    f = freqs(64)
    y, b = reference(x, pos, f, (64,), False)
    got = w.rotary_axes(dev(x), dev(pos[0]), dev(f)).cpu().numpy().astype(np.float64)
    assert (np.abs(got - y) <= b).all()
    assert np.array_equal(got[0], x[0].astype(np.float64))       # position 0 turns nothing


def test_values_at_the_ends_of_fp16():
    x, pos = inputs(64, 2, 64, 1, seed=2)
    x[:16] = np.where(np.arange(64) % 2, 65504, -65504).astype(np.float16)
    x[16:32] = np.float16(6e-8)
    x[32:40, :, 3] = np.inf
    x[40:48, :, 5] = np.nan
    f = freqs(32)
    got = w.rotary_axes(dev(x), dev(pos), dev(f)).cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        y, b = reference(x, pos, f, (32,), False)
    over = np.abs(y[:16]) > 65520
    fine = np.abs(y[:16]) < 65500
    assert (np.isinf(got[:16][over])).all()
    assert (np.abs(got[:16] - y[:16]) <= b[:16])[fine].all()
    assert (np.abs(got[16:32] - y[16:32]) <= b[16:32]).all()
    # what is not finite stays in its own pair
    touched = np.zeros((64,), bool)
    touched[[3, 35]] = True
    assert np.isfinite(got[32:40][..., ~touched]).all() and not np.isfinite(got[32:40][..., touched]).all()
    touched = np.zeros((64,), bool)
    touched[[5, 37]] = True
    assert np.isfinite(got[40:48][..., ~touched]).all() and np.isnan(got[40:48][..., touched]).all()


@pytest.mark.parametrize("T,heads,extra", [(1, 6, 16), (37, 10, 512), (200, 40, 1024)])
def test_strided_rows_and_in_place(T, heads, extra):
    D, sections = 128, (24, 20, 20)
    x, pos = inputs(T, heads, D, 3, seed=T)
    f = freqs(64)
    wide = torch.full((T, heads * D + extra), 7.0, dtype=torch.float16, device="cuda")
    rows = wide[:, :heads * D].view(T, heads, D) if extra % D == 0 and T == 1 else \
        wide.as_strided((T, heads, D), (heads * D + extra, D, 1))
    rows.copy_(dev(x))
    apart = w.rotary_axes(dev(x), dev(pos), dev(f), sections, True)
    assert torch.equal(w.rotary_axes(rows, dev(pos), dev(f), sections, True), apart)
    w.rotary_axes(rows, dev(pos), dev(f), sections, True, out=rows)
    assert torch.equal(rows, apart)
    if T > 1:
        assert bool((wide[:, heads * D:] == 7).all())


def test_no_tokens():
    f = dev(freqs(64))
    x = torch.empty((0, 4, 128), dtype=torch.float16, device="cuda")
    assert w.rotary_axes(x, torch.empty((1, 0), dtype=torch.int64, device="cuda"), f).shape == (0, 4, 128)


def test_turning_back_gives_the_input():
    """The turn's inverse (its gradient's formula) is the turn by the negative position."""
    x, pos = inputs(50, 4, 128, 1, seed=9)
    f = dev(freqs(64))
    y = w.rotary_axes(dev(x), dev(pos), f)
    back = w.rotary_axes(y, dev(-pos), f).cpu().numpy().astype(np.float64)
    a = np.abs(x.astype(np.float64))
    pair = a[..., :64] + a[..., 64:]
    # two roundings to fp16 and 16 u, each on values of at most the pair's norm
    tol = 2 * (HALF_ROUND * math.sqrt(2) + 8 * U) * np.concatenate((pair, pair), -1) + 4 * HALF_TINY
    assert (np.abs(back - x) <= tol).all()
