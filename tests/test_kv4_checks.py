"""The attention block refuses malformed arguments before anything reaches the GPU (no GPU needed)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from w4a8_int8_gemm_amd import ops  # noqa: E402
from w4a8_int8_gemm_amd._lib import CacheStruct  # noqa: E402

CHECK = r"must|shape|head|group|workspace|stride|sections|slots|dims|T=|page|values|one row"
A, MIS = 4096, 4098


@pytest.fixture
def cpu_ok(monkeypatch):
    monkeypatch.setattr(ops, "_DEVICE_TYPE", "cpu")


def f16(*s):
    return torch.zeros(s, dtype=torch.float16)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def i64(*s):
    return torch.zeros(s, dtype=torch.int64)


def cache(pages=4, heads=2, page=16, D=64, G=32):
    return w.KV4Cache.empty(pages, heads, page, D, G, device="cpu")


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="device tensor"):
        w.rotary_axes(f16(1, 2, 64), i64(1, 1), torch.ones(32))
    with pytest.raises(ValueError, match="device tensor"):
        cache()


@pytest.mark.parametrize("D,G", [(64, 16), (64, 128), (128, 16), (256, 32), (96, 32), (512, 128), (32, 32)])
def test_cache_geometry(cpu_ok, D, G):
    with pytest.raises(ValueError, match=CHECK):
        cache(D=D, G=G)


@pytest.mark.parametrize("page", [8, 17, 24, 1 << 21])
def test_page_sizes(cpu_ok, page):
    with pytest.raises(ValueError, match=CHECK):
        cache(pages=1, heads=1, page=page)


def test_cache_tensors(cpu_ok):
    c = cache()
    for k, ks, v, vs in [(c.k[:3].clone(), c.k_scale, c.v, c.v_scale), (c.k, c.k_scale[..., :1].clone(), c.v, c.v_scale),
                         (c.k, c.k_scale, c.v[..., :16].clone(), c.v_scale), (c.k[:0], c.k_scale[:0], c.v[:0], c.v_scale[:0]),
                         (c.k, c.k_scale, c.v, c.v_scale.transpose(1, 2))]:
        with pytest.raises(ValueError, match=CHECK):
            w.KV4Cache(k, ks, v, vs)
    with pytest.raises(TypeError):
        w.KV4Cache(c.k.float(), c.k_scale, c.v, c.v_scale)
    with pytest.raises(TypeError):
        w.KV4Cache(c.k, c.k_scale.double(), c.v, c.v_scale)


@pytest.mark.parametrize("kw,exc", [
    (dict(x=f16(2, 128)), ValueError),
    (dict(x=f16(2, 3, 64).float()), TypeError),
    (dict(x=f16(2, 64, 3).transpose(1, 2)), ValueError),
    (dict(positions=i64(2, 2)), ValueError),
    (dict(positions=i64(1, 3)), ValueError),
    (dict(positions=i32(1, 2)), TypeError),
    (dict(inv_freq=torch.ones(12)), ValueError),
    (dict(inv_freq=torch.ones(40)), ValueError),
    (dict(inv_freq=torch.ones(0)), ValueError),
    (dict(inv_freq=torch.ones(32).double()), TypeError),
    (dict(sections=(16, 15)), ValueError),
    (dict(sections=(40, -8)), ValueError),
    (dict(sections=(8, 8, 8, 8)), ValueError),
    (dict(sections=()), ValueError),
    (dict(out=f16(2, 3, 32)), ValueError),
    (dict(out=f16(3, 3, 64)), ValueError),
])
def test_rotary_arguments(cpu_ok, kw, exc):
    args = dict(x=f16(2, 3, 64), positions=i64(1, 2), inv_freq=torch.ones(32))
    args.update(kw)
    with pytest.raises(exc, match=CHECK):
        w.rotary_axes(**args)


@pytest.mark.parametrize("kw,exc", [
    (dict(k=f16(3, 2, 32)), ValueError),
    (dict(k=f16(3, 3, 64)), ValueError),
    (dict(v=f16(4, 2, 64)), ValueError),
    (dict(v=f16(3, 2, 64).bfloat16()), TypeError),
    (dict(v=f16(3, 64, 2).transpose(1, 2)), ValueError),
    (dict(slots=i64(4)), ValueError),
    (dict(slots=i32(3)), TypeError),
    (dict(cache=None), TypeError),
])
def test_write_and_read_arguments(cpu_ok, kw, exc):
    args = dict(k=f16(3, 2, 64), v=f16(3, 2, 64), slots=i64(3), cache=cache())
    args.update(kw)
    with pytest.raises(exc, match=CHECK):
        w.kv4_write(**args)
    if "slots" in kw and exc is TypeError or "cache" in kw:
        with pytest.raises(exc, match=CHECK):
            w.kv4_read(args["cache"], args["slots"])


def test_read_outputs(cpu_ok):
    with pytest.raises(ValueError, match=CHECK):
        w.kv4_read(cache(), i64(3), k=f16(2, 2, 64))
    with pytest.raises(TypeError, match=CHECK):
        w.kv4_read(cache(), i64(3), v=f16(3, 2, 64).float())


@pytest.mark.parametrize("kw,exc", [
    (dict(q=f16(3, 4, 128)), ValueError),
    (dict(q=f16(3, 3, 64)), ValueError),
    (dict(q=f16(3, 0, 64)), ValueError),
    (dict(q=f16(3, 4, 64).float()), TypeError),
    (dict(q=f16(4, 4, 64)), ValueError),                 # no q_starts: one row a sequence
    (dict(page_table=i64(3, 2)), TypeError),
    (dict(page_table=i32(3)), ValueError),
    (dict(kv_lens=i32(2)), ValueError),
    (dict(kv_lens=i64(3)), TypeError),
    (dict(q_starts=i32(3)), ValueError),
    (dict(q_starts=i64(4)), TypeError),
    (dict(out=f16(3, 4, 32)), ValueError),
    (dict(lse=torch.zeros(3, 2)), ValueError),
    (dict(lse=f16(3, 4)), TypeError),
    (dict(workspace=torch.zeros(0, dtype=torch.int8)), TypeError),
    (dict(cache=None), TypeError),
])
def test_attention_arguments(cpu_ok, kw, exc):
    args = dict(q=f16(3, 4, 64), cache=cache(), page_table=i32(3, 2), kv_lens=i32(3))
    args.update(kw)
    with pytest.raises(exc, match=CHECK):
        w.kv4_attention(**args)


# ---- the C entry points

def struct(**kw):
    d = dict(k=A, v=A, k_scale=A, v_scale=A, pages=4, kv_heads=2, page_size=16, head_dim=64, group_size=32)
    d.update(kw)
    return ctypes.byref(CacheStruct(*[d[n] for n, _ in CacheStruct._fields_]))


S = w.Status


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96), S.ERR_SHAPE), (dict(head_dim=0), S.ERR_SHAPE), (dict(group_size=0), S.ERR_SHAPE),
    (dict(group_size=128), S.ERR_SHAPE), (dict(head_dim=256), S.ERR_SHAPE), (dict(page_size=8), S.ERR_SHAPE),
    (dict(page_size=48), S.ERR_SHAPE), (dict(page_size=0), S.ERR_SHAPE), (dict(kv_heads=0), S.ERR_SHAPE),
    (dict(pages=0), S.ERR_INVALID_ARG), (dict(pages=-1), S.ERR_INVALID_ARG), (dict(k=None), S.ERR_INVALID_ARG),
    (dict(v_scale=None), S.ERR_INVALID_ARG), (dict(v=MIS), S.ERR_ALIGNMENT), (dict(k_scale=MIS), S.ERR_ALIGNMENT),
])
def test_cache_errors(kw, status):
    L = w.lib()
    c = struct(**kw)
    assert L.kv4_write(A, 128, A, 128, A, 1, c, None) == status
    assert L.kv4_read(c, A, 1, A, A, None) == status
    assert attention(cache=c) == status
    assert L.w4a8_last_error()


def test_null_cache():
    L = w.lib()
    assert L.kv4_write(A, 128, A, 128, A, 1, None, None) == S.ERR_INVALID_ARG
    assert L.kv4_read(None, A, 1, A, A, None) == S.ERR_INVALID_ARG
    assert attention(cache=None) == S.ERR_INVALID_ARG


@pytest.mark.parametrize("args,status", [
    ((A, 128, A, 128, A, -1), S.ERR_INVALID_ARG), ((None, 128, A, 128, A, 1), S.ERR_INVALID_ARG),
    ((A, 128, A, 128, None, 1), S.ERR_INVALID_ARG), ((A, 120, A, 128, A, 1), S.ERR_SHAPE),
    ((A, 128, A, 132, A, 1), S.ERR_SHAPE), ((MIS, 128, A, 128, A, 1), S.ERR_ALIGNMENT),
    ((A, 128, A, 128, MIS, 1), S.ERR_ALIGNMENT), ((None, 0, None, 0, None, 0), S.OK),
    ((A, 128, A, 128, A, 1 << 40), S.ERR_INVALID_ARG),
])
def test_write_errors(args, status):
    assert w.lib().kv4_write(*args, struct(), None) == status


@pytest.mark.parametrize("args,status", [
    ((A, -1, A, A), S.ERR_INVALID_ARG), ((None, 1, A, A), S.ERR_INVALID_ARG), ((A, 1, A, None), S.ERR_INVALID_ARG),
    ((A, 1, MIS, A), S.ERR_ALIGNMENT), ((None, 0, None, None), S.OK),
])
def test_read_errors(args, status):
    assert w.lib().kv4_read(struct(), *args, None) == status


def rotary(x=A, x_stride=256, pos=A, freq=A, T=2, heads=4, D=64, R=64, axes=1, sections=(32,), out=A, out_stride=256):
    arr = None if sections is None else (ctypes.c_int32 * len(sections))(*sections)
    return w.lib().rotary_axes(x, x_stride, pos, freq, T, heads, D, R, axes, arr, 0, out, out_stride, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), S.ERR_INVALID_ARG), (dict(heads=-1), S.ERR_INVALID_ARG), (dict(heads=1 << 20), S.ERR_INVALID_ARG),
    (dict(D=60), S.ERR_SHAPE), (dict(D=0), S.ERR_SHAPE), (dict(D=2048), S.ERR_SHAPE), (dict(R=24), S.ERR_SHAPE),
    (dict(R=0), S.ERR_SHAPE), (dict(R=128), S.ERR_SHAPE), (dict(axes=0), S.ERR_SHAPE), (dict(axes=4), S.ERR_SHAPE),
    (dict(sections=(31,)), S.ERR_SHAPE), (dict(axes=2, sections=(40, -8)), S.ERR_SHAPE),
    (dict(sections=None), S.ERR_INVALID_ARG), (dict(x=None), S.ERR_INVALID_ARG), (dict(out=None), S.ERR_INVALID_ARG),
    (dict(x_stride=248), S.ERR_SHAPE), (dict(out_stride=260), S.ERR_SHAPE), (dict(x_stride=264), S.ERR_INVALID_ARG),
    (dict(x=MIS), S.ERR_ALIGNMENT), (dict(pos=MIS), S.ERR_ALIGNMENT), (dict(T=0, x=None, out=None), S.OK),
])
def test_rotary_errors(kw, status):
    assert rotary(**kw) == status


def attention(q=A, stride=256, T=3, heads=4, cache=0, table=A, max_pages=2, lens=A, starts=A, B=3, max_q=2, causal=1,
              window=0, scale=1.0, out=A, lse=A, ws=256, ws_bytes=1 << 40):
    c = struct() if cache == 0 else cache
    return w.lib().kv4_attention(q, stride, T, heads, c, table, max_pages, lens, starts, B, max_q, causal, window, scale,
                                 out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), S.ERR_INVALID_ARG), (dict(B=-1), S.ERR_INVALID_ARG), (dict(max_q=-1), S.ERR_INVALID_ARG),
    (dict(max_pages=-1), S.ERR_INVALID_ARG), (dict(heads=0), S.ERR_INVALID_ARG), (dict(heads=3), S.ERR_SHAPE),
    (dict(max_pages=1 << 28), S.ERR_SHAPE), (dict(window=-1), S.ERR_INVALID_ARG),
    (dict(window=4, causal=0), S.ERR_INVALID_ARG), (dict(scale=0.0), S.ERR_INVALID_ARG),
    (dict(scale=float("nan")), S.ERR_INVALID_ARG), (dict(scale=float("inf")), S.ERR_INVALID_ARG),
    (dict(starts=None, B=2), S.ERR_SHAPE), (dict(starts=None, max_q=0), S.ERR_SHAPE), (dict(B=0), S.ERR_SHAPE),
    (dict(q=None), S.ERR_INVALID_ARG), (dict(out=None), S.ERR_INVALID_ARG), (dict(table=None), S.ERR_INVALID_ARG),
    (dict(lens=None), S.ERR_INVALID_ARG), (dict(stride=248), S.ERR_SHAPE), (dict(stride=260), S.ERR_SHAPE),
    (dict(q=MIS), S.ERR_ALIGNMENT), (dict(out=MIS), S.ERR_ALIGNMENT), (dict(lens=MIS), S.ERR_ALIGNMENT),
    (dict(T=0, q=None, out=None), S.OK),
])
def test_attention_errors(kw, status):
    assert attention(**kw) == status
