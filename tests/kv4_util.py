"""The attention block's operators from their definitions, in 64 bits on the CPU.

Nothing here is shared with the library: the cache's format, the int4 rule,
rotary positions and attention are written again from include/w4a8.h.
"""
import math

import numpy as np

HALF_ROUND = 2.0 ** -11          # half a step of fp16, relative
HALF_TINY = 2.0 ** -25           # half a step of its subnormals
U = 2.0 ** -24                   # half a step of fp32, relative

HEADS_AND_GROUPS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 64), (256, 128), (256, 256)]


def int4_rule(x, group):
    """fp16 [..., d] -> (codes int [..., d], scales fp32 [..., d / group]); the quotient rounded to
    fp32 as the rule says (a 64-bit quotient rounded again to 32 is the correctly rounded one)."""
    g = x.astype(np.float64).reshape(*x.shape[:-1], x.shape[-1] // group, group)
    s = (np.abs(g).max(-1) / 7).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(s[..., None] > 0, g / s[..., None].astype(np.float64), 0.0).astype(np.float32)
    t = t.astype(np.float64)
    q = np.clip(np.sign(t) * np.floor(np.abs(t) + 0.5), -7, 7).astype(np.int64)
    return q.reshape(x.shape), s


def row_bytes(codes, kind):
    """Codes [..., d] to the stored bytes of a K or V row: word b n + g is natural word 4 g + b
    of a K row, byte r n + g natural byte 16 g + r of a V row (n = d / 32)."""
    u = (codes & 15).astype(np.uint8)
    nat = u[..., 0::2] | (u[..., 1::2] << 4)
    out = np.empty_like(nat)
    n = codes.shape[-1] // 32
    for j in range(nat.shape[-1]):
        g, r = divmod(j, 16)
        at = (r // 4 * n + g) * 4 + r % 4 if kind == "k" else r * n + g
        out[..., at] = nat[..., j]
    return out


def row_codes(stored, kind):
    """The inverse of row_bytes."""
    d = 2 * stored.shape[-1]
    n = d // 32
    codes = np.empty((*stored.shape[:-1], d), np.int64)
    for j in range(d // 2):
        g, r = divmod(j, 16)
        at = (r // 4 * n + g) * 4 + r % 4 if kind == "k" else r * n + g
        for half in (0, 1):
            u = (stored[..., at].astype(np.int64) >> (4 * half)) & 15
            codes[..., 2 * j + half] = u - 16 * (u > 7)
    return codes


def values(codes, scale, group):
    """fp64 values code * scale."""
    return codes.astype(np.float64) * np.repeat(scale.astype(np.float64), group, -1)


def visible(n, m, i, causal, window):
    """The keys query i of m sees of n: a range (lo, hi)."""
    if not causal:
        return 0, n
    hi = n - m + i + 1
    lo = max(0, hi - window) if window else 0
    return lo, max(hi, lo if hi > 0 else 0) if hi > 0 else 0


def attention(q, k, v, there, m_of, n_of, causal, window, scale, page_size):
    """Rows of one sequence: q fp16 [m, hq, d], k and v fp64 [n, hk, d], there bool [n].
    -> (out, lse, bound of out, bound of lse), all fp64.

    The bounds count roundings.  A score is a sum of d products of fp16 and 4-bit values (exact)
    in fp32, scaled twice: (d + 8) steps of 2 u on scale * sum |q k| (2 u for a product sum whose
    internal rounding may be a truncation).  exp2 of a score holds that error plus a few steps; the
    weights are rounded to fp16 once (2^-11); sums over n keys add n u.  Sum and output are joined
    over parts of the keys with a few more steps each."""
    m, hq, d = q.shape
    n, hk = k.shape[:2]
    out = np.zeros((m, hq, d))
    lse = np.full((m, hq), -math.inf)
    out_b = np.full((m, hq, d), HALF_TINY)
    lse_b = np.zeros((m, hq))
    for i in range(m):
        if causal:
            hi = n - m + i + 1
            lo = max(0, hi - window) if window else 0
        else:
            lo, hi = 0, n
        if hi <= lo:
            continue
        ok = there[lo:hi]
        if not ok.any():
            continue
        kk, vv = k[lo:hi][ok], v[lo:hi][ok]
        for h in range(hq):
            g = h // (hq // hk)
            qq = q[i, h].astype(np.float64)
            s = kk[:, g] @ qq * scale
            reach = (np.abs(kk[:, g]) @ np.abs(qq)).max() * scale
            top = s.max()
            e = np.exp(s - top)
            tot = e.sum()
            p = e / tot
            out[i, h] = p @ vv[:, g]
            lse[i, h] = top + math.log(tot)
            ds = (d + 8) * 2 * U * reach + 8 * U
            count = len(s) * U + 64 * U
            out_b[i, h] += HALF_ROUND * np.abs(out[i, h]) * 1.01 + \
                (HALF_ROUND + 2 * ds + 2 * count) * 1.01 * (p @ np.abs(vv[:, g]))
            lse_b[i, h] = ds + count + 8 * U * abs(lse[i, h])
    return out, lse, out_b, lse_b
