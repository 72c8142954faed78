"""Arguments of the attention block at the ends of their ranges (no GPU needed)."""
import ctypes
import subprocess

import pytest

pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.test_kv4_checks import MIS, S, attention, cache, cpu_ok, f16, i32, i64, struct  # noqa: E402,F401


@pytest.mark.parametrize("scale", [2.0 ** 127 * 1.01, 3e38, 3.4e38])
def test_scales_whose_exponent_leaves_fp32(scale):
    """scale * log2(e) has to be finite."""
    assert attention(scale=scale) == S.ERR_INVALID_ARG
    assert attention(scale=2.0 ** 127, q=MIS) == S.ERR_ALIGNMENT      # taken; what is refused comes later
    assert w.lib().w4a8_last_error()


class Recorder:
    """The C library's kv4_attention, its numbers kept instead of run."""

    def __init__(self, monkeypatch):
        from w4a8_int8_gemm_amd import kv4
        real = w.lib()
        rec = self

        class Lib:
            kv4_attention_workspace_size = staticmethod(real.kv4_attention_workspace_size)
            kv4_attention = "kv4_attention"

        monkeypatch.setattr(kv4, "lib", Lib)
        monkeypatch.setattr(kv4, "_call", lambda index, fn, *args: setattr(rec, "args", (fn, args)))


@pytest.mark.parametrize("given,passed", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                          (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 70, 2 ** 31 - 1), (-1, -1), (-2 ** 32 + 5, -1)])
def test_windows_past_32_bits(cpu_ok, monkeypatch, given, passed):
    """A window longer than any cache hides nothing; it is not taken modulo 2^32."""
    r = Recorder(monkeypatch)
    w.kv4_attention(f16(3, 4, 64), cache(), i32(3, 2), i32(3), window=given)
    fn, args = r.args
    at = w._lib._SIGNATURES[fn]
    assert len(args) + 1 == len(at) and ctypes.c_int32(args[12]).value == args[12] == passed


@pytest.mark.parametrize("given,passed", [(2, 2), (50, 3), (2 ** 32 + 1, 3), (2 ** 70, 3), (-2 ** 32 + 1, -1)])
def test_max_q_past_32_bits(cpu_ok, monkeypatch, given, passed):
    r = Recorder(monkeypatch)
    w.kv4_attention(f16(3, 4, 64), cache(), i32(1, 2), i32(1), q_starts=i32(2), max_q=given)
    assert r.args[1][10] == passed
    size = w.kv4_attention_workspace_size
    assert size(4, 2, 64, 3, 1, given) == size(4, 2, 64, 3, 1, passed)


@pytest.mark.parametrize("bad", [None, [[0, 1]], 3])
def test_what_is_no_tensor_is_named(cpu_ok, bad):
    import torch
    c = cache()
    calls = [lambda: w.rotary_axes(bad, i64(1, 2), torch.ones(32)), lambda: w.rotary_axes(f16(2, 3, 64), bad, torch.ones(32)),
             lambda: w.rotary_axes(f16(2, 3, 64), i64(1, 2), bad), lambda: w.kv4_write(f16(3, 2, 64), f16(3, 2, 64), bad, c),
             lambda: w.kv4_write(bad, f16(3, 2, 64), i64(3), c), lambda: w.kv4_read(c, bad),
             lambda: w.kv4_attention(f16(3, 4, 64), c, bad, i32(3)), lambda: w.kv4_attention(f16(3, 4, 64), c, i32(3, 2), bad),
             lambda: w.KV4Cache(bad, c.k_scale, c.v, c.v_scale), lambda: w.KV4Cache(c.k, bad, c.v, c.v_scale)]
    for call in calls:
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            call()
    if bad is not None:
        for kw in (dict(q_starts=bad), dict(workspace=bad), dict(out=bad), dict(lse=bad)):
            with pytest.raises(TypeError, match="must be a torch.Tensor"):
                w.kv4_attention(f16(3, 4, 64), c, i32(3, 2), i32(3), **kw)


@pytest.mark.parametrize("kw", [dict(B=1 << 20, T=1 << 20, starts=None, max_q=1, heads=16), dict(B=1 << 20, T=1 << 20, heads=32),
                                dict(B=1 << 20, T=1 << 20, max_q=1, heads=16 * 33)])
def test_more_workgroups_than_a_launch_holds(kw):
    """2^24 workgroups of 256 threads would wrap at 2^32 threads without an error."""
    heads = kw["heads"]
    c = struct(kv_heads=16)
    assert attention(cache=c, stride=heads * 64, **kw) == S.ERR_INVALID_ARG
    assert b"workgroups" in w.lib().w4a8_last_error()
    kw = dict(kw, B=1 << 16, T=1 << 16, max_q=1)
    assert attention(cache=c, stride=heads * 64, ws_bytes=0, **kw) == S.ERR_WORKSPACE    # taken; refused later


def test_no_entry_point_can_throw_for_want_of_random_numbers():
    """std::random_device throws where its source cannot be read, through a C entry point."""
    out = subprocess.run(["nm", "-D", "--undefined-only", w.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert "random_device" not in out and "__cxa_throw" not in out
