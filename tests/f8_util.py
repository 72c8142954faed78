"""8-bit floating point in blocks of 128 and the norm from their definitions, in
64 bits on the CPU, with bounds that count the roundings of include/w4a8.h.

Nothing here is shared with the library."""
import math

import numpy as np

U = 2.0 ** -24                   # half a step of fp32, relative
HALF_ROUND = 2.0 ** -11          # half a step of fp16, relative
HALF_TINY = 2.0 ** -25           # half a step of its subnormals
F8_ROUND = 2.0 ** -4             # half a step of e4m3, relative
F8_TINY = 2.0 ** -10             # half a step of its subnormals
BLOCK = 128


def decode(codes):
    """e4m3 codes (uint8) to fp64; 0x7f and 0xff are NaN."""
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9.0)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def encode(t):
    """fp values in [-448, 448] to the nearest e4m3 code, ties to the even one: by search over the values."""
    grid = decode(np.arange(127, dtype=np.uint8))
    a = np.abs(t.astype(np.float64))
    hi = np.minimum(np.searchsorted(grid, a), 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = grid[hi] - a, a - grid[lo]
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return pick | (np.signbit(t).astype(np.uint8) << 7)


def _padded(x, rows):
    r, c = x.shape
    return np.pad(x, ((0, -r % rows), (0, -c % BLOCK)))


def rule(x, rows):
    """fp16 [R, C] in blocks of rows x 128: (codes uint8 [R, C], scales fp32 [R', C']).  The quotient is
    taken in 64 bits and rounded to 32, which is the correctly rounded one; finite input."""
    p = _padded(x.astype(np.float64), rows)
    b = p.reshape(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)
    s = (np.abs(b).max((1, 3), keepdims=True) / 448).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(s > 0, b / s.astype(np.float64), 0.0).astype(np.float32)
    q = encode(t).reshape(p.shape)[:x.shape[0], :x.shape[1]]
    return np.ascontiguousarray(q), s[:, 0, :, 0]


def spread(scale, rows, shape):
    """Block scales [R', C'] to every element of `shape`, fp64."""
    return np.repeat(np.repeat(scale.astype(np.float64), rows, 0), BLOCK, 1)[:shape[0], :shape[1]]


def _exponents(codes):
    """The exponent a code is aligned by: that of its field, -6 for subnormals and zeros."""
    return np.maximum(((codes.astype(np.int64) >> 3) & 15) - 7, -6)


def product(xq, sx, wq, sw):
    """xq uint8 [M, K], sx [KB, M], wq uint8 [N, K], sw [NB, KB] -> (fp64 [M, N], bound of an fp32
    accumulation's distance from it).

    The bound: of eight consecutive products aligned to the largest exponent e, seven may lose what lies
    below 2^(e - 13); the groups' sums and the blocks are added in fp32 (2 U a step for an addition that may
    truncate), the two scales are multiplied in fp32."""
    M, K = xq.shape
    N = wq.shape[0]
    xv, wv = decode(xq), decode(wq)
    KB = -(-K // BLOCK)
    out, bound, reach = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    ex, ew = _exponents(xq), _exponents(wq)
    for b in range(KB):
        k = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        s = sx[b].astype(np.float64)[:, None] * np.repeat(sw[:, b].astype(np.float64), BLOCK)[:N]
        out += (xv[:, k] @ wv[:, k].T) * s
        reach += (np.abs(xv[:, k]) @ np.abs(wv[:, k]).T) * np.abs(s)
        loss = np.zeros((M, N))
        for at in range(k.start, k.stop, 8):
            e = (ex[:, None, at:at + 8] + ew[None, :, at:at + 8]).max(-1)
            loss += 7 * 2.0 ** (e - 13.0)
        bound += loss * np.abs(s)
    return out, bound + (KB + 40) * 2 * U * reach


def activation(g, kind):
    if kind == "silu":
        with np.errstate(over="ignore"):
            return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def gated(xq, sx, wg, sg, wu, su, kind):
    """(act(g) u in fp64, bound of its fp32 value).  The slope of silu and of gelu lies below 1.13; the
    activation's exponential and reciprocal are good to 2^-20 of it for |g| <= 60."""
    g, dg = product(xq, sx, wg, sg)
    u, du = product(xq, sx, wu, su)
    assert np.abs(g).max(initial=0) <= 60
    a = activation(g, kind)
    da = 1.13 * dg + 2.0 ** -20 * np.abs(a)
    return a * u, da * (np.abs(u) + du) + np.abs(a) * du + 2 * U * np.abs(a * u)


def fp16_bound(v, dv):
    return dv + (np.abs(v) + dv) * HALF_ROUND * 1.001 + HALF_TINY


def check_codes_f8(codes, scale, v, dv, what=""):
    """codes uint8 [M, N] and scale fp32 [NB, M] against v [M, N] known up to dv."""
    M, N = v.shape
    for b in range(-(-N // BLOCK)):
        n = slice(b * BLOCK, min(N, (b + 1) * BLOCK))
        top = np.abs(v[:, n]).max(1)
        s = scale[b].astype(np.float64)
        ds = dv[:, n].max(1) / 448 + 2 * U * top / 448
        assert (np.abs(s - top / 448) <= ds * 1.001 + 2.0 ** -126).all(), f"{what}: scales of block {b}"
        got = decode(codes[:, n]) * s[:, None]
        # half a step of the code, of the value or below 2^-6 of the scale's unit; the quotient's rounding
        b_ = np.abs(v[:, n]) * (F8_ROUND + 4 * U) * 1.001 + F8_TINY * s[:, None] * 1.001 + dv[:, n] * 1.1 + 448 * ds[:, None] * F8_ROUND
        assert (np.abs(got - v[:, n]) <= b_).all(), f"{what}: codes of block {b}"


def norm(x, gain, eps, residual=None):
    """(v fp64, its bound, h fp64)."""
    h = x.astype(np.float64)
    if residual is not None:
        h = h + residual.astype(np.float64)
    K = h.shape[1]
    mean = (h * h).mean(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(mean > 0, h / np.sqrt(mean + eps), 0.0) * gain.astype(np.float64)
    # squares of rounded h, at most K / 64 + 24 additions in a row, halved by the root; then the root, the
    # quotient, two products and h's own rounding
    rel = ((K / 64 + 28) / 2 + 8) * U
    return v, rel * np.abs(v), h
