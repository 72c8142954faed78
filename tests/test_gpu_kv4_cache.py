"""Writing the 4-bit cache and reading it back on the GPU: bit for bit the int4 rule."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.kv4_util import HEADS_AND_GROUPS, int4_rule, row_bytes, row_codes, values  # noqa: E402

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make(pages, heads, page, D, G, fill=0xA5):
    c = w.KV4Cache.empty(pages, heads, page, D, G)
    c.k.fill_(fill)
    c.v.fill_(fill)
    c.k_scale.fill_(float("nan"))
    c.v_scale.fill_(float("nan"))
    return c


def rows_of(c, kind):
    """All slots' rows: (bytes [slots, heads, D/2], scales [slots, heads, groups])."""
    b, s = (c.k, c.k_scale) if kind == "k" else (c.v, c.v_scale)
    b, s = b.cpu().numpy(), s.cpu().numpy()
    return (b.transpose(0, 2, 1, 3).reshape(-1, c.kv_heads, c.head_dim // 2),
            s.transpose(0, 2, 1, 3).reshape(-1, c.kv_heads, c.head_dim // c.group_size))


def data(T, heads, D, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((2, T, heads, D)).astype(np.float16)
    x[:, :, :, 3::29] *= 8
    if T > 3:
        x[0, 1] = 0                                        # an all-zero token
        x[1, 2, :, :D // 2] = 0
        x[0, 3] = np.float16(6e-8) * r.integers(-3, 4, (heads, D))
    if T > 5:
        x[1, 4] = r.choice([-65504, 65504, 1], (heads, D)).astype(np.float16)
        x[0, 5] = (np.arange(D) % 15 - 7) / 2             # quotients at and next to halves
    return x[0], x[1]


@pytest.mark.parametrize("D,G", HEADS_AND_GROUPS)
@pytest.mark.parametrize("T,heads,page", [(1, 1, 16), (3, 5, 32), (70, 3, 64), (515, 8, 16)])
def test_write_and_read(D, G, T, heads, page):
    k, v = data(T, heads, D, seed=T + D + G)
    pages = T // page + 4
    c = make(pages, heads, page, D, G)
    r = np.random.default_rng(T)
    slots = r.permutation(pages * page)[:T].astype(np.int64)
    w.kv4_write(dev(k), dev(v), dev(slots), c)
    for kind, x in (("k", k), ("v", v)):
        q, s = int4_rule(x, G)
        b, sc = rows_of(c, kind)
        assert np.array_equal(b[slots], row_bytes(q, kind))
        assert np.array_equal(sc[slots], s)
        rest = np.setdiff1d(np.arange(pages * page), slots)
        assert (b[rest] == 0xA5).all() and np.isnan(sc[rest]).all()      # nothing else is touched
    kk, vv = w.kv4_read(c, dev(slots))
    for got, x in ((kk, k), (vv, v)):
        q, s = int4_rule(x, G)
        want = (q.astype(np.float32) * np.repeat(s, G, -1)).astype(np.float16)
        assert np.array_equal(got.cpu().numpy(), want)


def test_agrees_with_the_weight_packers_oracle(oracle):
    x = np.random.default_rng(5).standard_normal((40, 128)).astype(np.float16)
    for G in (64, 128):
        c = make(3, 1, 16, 128, G)
        t = dev(x[:, None, :])
        w.kv4_write(t, t, torch.arange(40, device="cuda"), c)
        packed, s = oracle.pack_weight_int4(x, G)
        b, sc = rows_of(c, "k")
        nat = np.stack((packed & 15, packed >> 4), -1).reshape(40, 128).astype(np.int64)
        assert np.array_equal(row_codes(b[:40, 0], "k") & 15, nat)
        assert np.array_equal(sc[:40, 0], s)


def test_slots_outside_the_cache_are_skipped():
    k, v = data(8, 2, 64, seed=1)
    k[[1, 4]], v[[1, 4]] = np.nan, np.inf                  # padding rows hold anything
    c = make(2, 2, 16, 64, 32)
    slots = np.array([0, -1, 31, 5, 32, 2 ** 40, -2 ** 62, 17], np.int64)
    w.kv4_write(dev(k), dev(v), dev(slots), c)
    b, sc = rows_of(c, "v")
    for t, s in enumerate(slots):
        if 0 <= s < 32:
            q, want = int4_rule(v[t], 32)
            assert np.array_equal(b[s], row_bytes(q, "v")) and np.array_equal(sc[s], want)
    rest = np.setdiff1d(np.arange(32), slots)
    assert (b[rest] == 0xA5).all() and np.isnan(sc[rest]).all()
    kk, vv = w.kv4_read(c, dev(slots))
    out = (slots < 0) | (slots >= 32)
    assert bool((kk[dev(out)] == 0).all()) and bool((vv[dev(out)] == 0).all())
    q, s = int4_rule(k[~out], 32)
    assert np.array_equal(kk.cpu().numpy()[~out], values(q, s, 32).astype(np.float32).astype(np.float16))


def test_strided_rows_of_the_qkv_product():
    T, hq, hk, D = 45, 8, 2, 128
    qkv = torch.randn(T, hq + 2 * hk, D, device="cuda").half()
    slots = torch.randperm(64, device="cuda")[:T].contiguous()
    a, b = make(4, hk, 16, D, 64), make(4, hk, 16, D, 64)
    w.kv4_write(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, a)
    w.kv4_write(qkv[:, hq:hq + hk].contiguous(), qkv[:, hq + hk:].contiguous(), slots, b)
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale[:], b.k_scale), (a.v_scale, b.v_scale)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_offsets_past_32_bits():
    """A cache whose buffers are over 4 GiB each: the last slots are written and read."""
    D, G, page, heads = 256, 64, 1 << 12, 8
    pages = (4 << 30) // (page * heads * D // 2) + 3
    c = w.KV4Cache.empty(pages, heads, page, D, G)
    assert c.k.numel() > 1 << 32
    T = 37
    k, v = data(T, heads, D, seed=3)
    slots = np.arange(pages * page - T, pages * page, dtype=np.int64)
    w.kv4_write(dev(k), dev(v), dev(slots), c)
    kk, vv = w.kv4_read(c, dev(slots))
    for got, x in ((kk, k), (vv, v)):
        q, s = int4_rule(x, G)
        assert np.array_equal(got.cpu().numpy(), (q.astype(np.float32) * np.repeat(s, G, -1)).astype(np.float16))
    q, s = int4_rule(k, G)
    assert np.array_equal(c.k[-1, :, -T:].cpu().numpy().transpose(1, 0, 2), row_bytes(q, "k"))


def test_no_tokens_and_another_stream():
    c = make(1, 2, 16, 64, 64)
    none = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    at = torch.empty((0,), dtype=torch.int64, device="cuda")
    w.kv4_write(none, none, at, c)
    assert w.kv4_read(c, at)[0].shape == (0, 2, 64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        x = torch.randn(16, 2, 64, device="cuda").half()
        w.kv4_write(x, x, torch.arange(16, device="cuda"), c)
        k, v = w.kv4_read(c, torch.arange(16, device="cuda"))
    st.synchronize()
    q, s = int4_rule(x.cpu().numpy(), 64)
    want = (q.astype(np.float32) * np.repeat(s, 64, -1)).astype(np.float16)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want)
