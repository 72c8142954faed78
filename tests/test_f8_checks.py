"""What the 8-bit floating point operators and the norm refuse, before anything reaches a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from w4a8_int8_gemm_amd import ops  # noqa: E402

P = ctypes.c_void_p
A, A2, A3, A4, A5, A6, A7 = (P(4096 * i) for i in range(1, 8))
MIS, MIS4 = P(4096 + 8), P(4096 + 2)
S = w.Status


@pytest.mark.parametrize("call,status", [
    # quantize_act_f8(x, M, K, xq, scale, stream)
    (lambda L: L.quantize_act_f8(A, 4, 12, A2, A3, None), S.ERR_SHAPE),
    (lambda L: L.quantize_act_f8(A, 4, 0, A2, A3, None), S.ERR_SHAPE),
    (lambda L: L.quantize_act_f8(A, -1, 16, A2, A3, None), S.ERR_INVALID_ARG),
    (lambda L: L.quantize_act_f8(A, (1 << 25) + 1, 16, A2, A3, None), S.ERR_INVALID_ARG),
    (lambda L: L.quantize_act_f8(A, 4, 16, None, A3, None), S.ERR_INVALID_ARG),
    (lambda L: L.quantize_act_f8(MIS, 4, 16, A2, A3, None), S.ERR_ALIGNMENT),
    (lambda L: L.quantize_act_f8(A, 4, 16, A2, MIS4, None), S.ERR_ALIGNMENT),
    (lambda L: L.quantize_act_f8(None, 0, 16, None, None, None), S.OK),
    # quantize_weight_f8(w, N, K, wq, scale, stream)
    (lambda L: L.quantize_weight_f8(A, 4, 20, A2, A3, None), S.ERR_SHAPE),
    (lambda L: L.quantize_weight_f8(A, 1 << 30, 1 << 20, A2, A3, None), S.ERR_SHAPE),
    (lambda L: L.quantize_weight_f8(A, 4, 16, A2, None, None), S.ERR_INVALID_ARG),
    (lambda L: L.quantize_weight_f8(None, 0, 16, None, None, None), S.OK),
    # rmsnorm_quant(mode, x, residual, gain, eps, M, K, gs, q, scale, residual_out, stream)
    (lambda L: L.rmsnorm_quant(4, A, None, A2, 1e-6, 4, 256, 0, A3, A4, None, None), S.ERR_INVALID_ARG),
    (lambda L: L.rmsnorm_quant(3, A, None, A2, 1e-6, 4, 250, 0, A3, A4, None, None), S.ERR_SHAPE),
    (lambda L: L.rmsnorm_quant(3, A, None, A2, -1e-6, 4, 256, 0, A3, A4, None, None), S.ERR_INVALID_ARG),
    (lambda L: L.rmsnorm_quant(3, A, None, A2, float("nan"), 4, 256, 0, A3, A4, None, None), S.ERR_INVALID_ARG),
    (lambda L: L.rmsnorm_quant(3, A, None, A2, float("inf"), 4, 256, 0, A3, A4, None, None), S.ERR_INVALID_ARG),
    (lambda L: L.rmsnorm_quant(1, A, None, A2, 1e-6, 4, 256, 32, A3, A4, None, None), S.ERR_SHAPE),
    (lambda L: L.rmsnorm_quant(1, A, None, A2, 1e-6, 4, 192, 128, A3, A4, None, None), S.ERR_SHAPE),
    (lambda L: L.rmsnorm_quant(0, A, None, None, 1e-6, 4, 256, 0, A3, A4, None, None), S.ERR_INVALID_ARG),
    (lambda L: L.rmsnorm_quant(0, A, None, A2, 1e-6, 4, 256, 0, A3, None, None, None), S.ERR_INVALID_ARG),
    (lambda L: L.rmsnorm_quant(0, A, MIS, A2, 1e-6, 4, 256, 0, A3, A4, None, None), S.ERR_ALIGNMENT),
    (lambda L: L.rmsnorm_quant(0, A, A5, A2, 1e-6, 4, 256, 0, A3, A4, MIS, None), S.ERR_ALIGNMENT),
    (lambda L: L.rmsnorm_quant(0, A, A5, A2, 1e-6, (1 << 25) + 1, 256, 0, A3, A4, A6, None), S.ERR_INVALID_ARG),
    (lambda L: L.rmsnorm_quant(0, A, A5, A2, 1e-6, 4, (1 << 22) + 8, 0, A3, A4, A6, None), S.ERR_INVALID_ARG),
    (lambda L: L.rmsnorm_quant(0, None, None, None, 1e-6, 0, 256, 0, None, None, None, None), S.OK),
    # f8_gemm(xq, sx, wq, sw, y, M, N, K, ws, bytes, stream)
    (lambda L: L.f8_gemm(A, A2, A3, A4, A5, 4, 8, 24, None, 0, None), S.ERR_SHAPE),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A5, 4, 8, 0, None, 0, None), S.ERR_SHAPE),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A5, 4, 8, (1 << 22) + 16, None, 0, None), S.ERR_SHAPE),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A5, 4, -8, 128, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A5, (1 << 25) + 1, 8, 128, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A5, 4, (1 << 27) + 1, 128, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A5, 1 << 25, 1 << 27, 128, None, 0, None), S.ERR_SHAPE),
    (lambda L: L.f8_gemm(A, None, A3, A4, A5, 4, 8, 128, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm(A, A2, A3, A4, None, 4, 8, 128, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm(A, A2, MIS, A4, A5, 4, 8, 128, None, 0, None), S.ERR_ALIGNMENT),
    (lambda L: L.f8_gemm(A, A2, A3, MIS4, A5, 4, 8, 128, None, 0, None), S.ERR_ALIGNMENT),
    (lambda L: L.f8_gemm(A, A2, A3, A4, MIS, 4, 8, 128, None, 0, None), S.ERR_ALIGNMENT),
    (lambda L: L.f8_gemm(None, None, None, None, None, 0, 8, 128, None, 0, None), S.OK),
    (lambda L: L.f8_gemm(None, None, None, None, None, 4, 0, 128, None, 0, None), S.OK),
    # f8_gemm_gated(xq, sx, wg, sg, wu, su, act, M, N, K, y, yq, ys, ws, bytes, stream)
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, A5, A6, 2, 4, 8, 128, A7, None, None, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, None, A6, 0, 4, 8, 128, A7, None, None, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, A5, A6, 0, 4, 8, 128, None, None, None, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, A5, A6, 0, 4, 8, 128, A7, A7, None, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, A5, A6, 0, 4, 8, 128, None, A7, None, None, 0, None), S.ERR_INVALID_ARG),
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, A5, A6, 0, 4, 8, 128, None, MIS, A7, None, 0, None), S.ERR_ALIGNMENT),
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, MIS, A6, 0, 4, 8, 128, A7, None, None, None, 0, None), S.ERR_ALIGNMENT),
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, A5, A6, 0, 4, 8, 40, A7, None, None, None, 0, None), S.ERR_SHAPE),
    (lambda L: L.f8_gemm_gated(None, None, None, None, None, None, 1, 4, 0, 128, None, None, None, None, 0, None), S.OK),
    # linear in the F8 mode
    (lambda L: L.linear(3, A, 4, 256, A2, A3, 0, 8, A4, None, 0, None), S.ERR_WORKSPACE),
    (lambda L: L.linear(3, A, 4, 256, A2, A3, 0, 8, A4, P(4096 + 16), 1 << 30, None), S.ERR_WORKSPACE),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A, 5, 500, 8208, None, 0, None), S.ERR_WORKSPACE),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A, 300, 200, 4112, None, 0, None), S.ERR_WORKSPACE),
    (lambda L: L.f8_gemm(A, A2, A3, A4, A, 300, 200, 4112, A, L.f8_gemm_workspace_size(300, 200, 4112) - 1, None),
     S.ERR_WORKSPACE),
    (lambda L: L.f8_gemm_gated(A, A2, A3, A4, A3, A4, 0, 130, 300, 4112, None, A, A2, None, 0, None), S.ERR_WORKSPACE),
    (lambda L: L.linear(3, A, 4, 264, A2, A3, 0, 8, A4, A5, 1 << 30, None), S.ERR_SHAPE),
    (lambda L: L.linear(3, A, 4, 256, A2, A3, 0, 8, None, A5, 1 << 30, None), S.ERR_INVALID_ARG),
    (lambda L: L.linear(3, A, 0, 256, A2, A3, 0, 8, A4, None, 0, None), S.OK),
])
def test_refused_before_the_device(call, status):
    got = call(w.lib())
    assert got == int(status), (got, status, w.lib().w4a8_last_error())
    if status != S.OK:
        assert w.lib().w4a8_last_error().decode()


M, N, K = 5, 200, 272
KB, NB = 3, 2
E = torch.float8_e4m3fn


@pytest.fixture
def cpu_ok(monkeypatch):
    monkeypatch.setattr(ops, "_DEVICE_TYPE", "cpu")


def f8(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(E)


def f32(*shape):
    return torch.ones(shape)


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def test_host_tensors():
    with pytest.raises(ValueError, match="device"):
        w.f8_gemm(f8(M, K), f32(KB, M), f8(N, K), f32(NB, KB))
    with pytest.raises(ValueError, match="device"):
        w.rmsnorm_quant(w.Mode.F8, f16(M, K), f16(K))
    with pytest.raises(ValueError, match="device"):
        w.quantize_act_f8(f16(M, K))


@pytest.mark.parametrize("args,exc", [
    ((f8(M, K), f32(M, KB), f8(N, K), f32(NB, KB)), ValueError),        # scales of a token side by side
    ((f8(M, K), f32(KB - 1, M), f8(N, K), f32(NB, KB)), ValueError),    # the short block's scales missing
    ((f8(M, K), f32(KB, M), f8(N, K), f32(N, KB)), ValueError),         # a scale for each weight row
    ((f8(M, K), f32(KB, M), f8(N, K), f32(KB, NB)), ValueError),        # transposed
    ((f8(M, K), f32(KB, M), f8(N, K + 16), f32(NB, KB)), ValueError),   # another K
    ((f8(M, K), f32(KB, M).double(), f8(N, K), f32(NB, KB)), TypeError),
    ((f16(M, K), f32(KB, M), f8(N, K), f32(NB, KB)), TypeError),
    ((f8(M, K), f32(KB, M), torch.zeros(N, K, dtype=torch.int8), f32(NB, KB)), TypeError),
    ((f8(M, K, 1), f32(KB, M), f8(N, K), f32(NB, KB)), ValueError),
    ((f8(K, M).t(), f32(KB, M), f8(N, K), f32(NB, KB)), ValueError),    # another order of the elements
    ((None, f32(KB, M), f8(N, K), f32(NB, KB)), TypeError),
    ((f8(M, K), None, f8(N, K), f32(NB, KB)), TypeError),
])
def test_product_operands(cpu_ok, args, exc):
    with pytest.raises(exc, match="must"):
        w.f8_gemm(*args)
    more = (f8(N, K), f32(NB, KB))
    with pytest.raises(exc, match="must"):
        w.f8_gemm_gated(*args, *more)
    if args[0] is not None and args[0].shape == (M, K) and args[0].is_contiguous() and args[0].dtype == E and \
            args[1] is not None and args[1].shape == (KB, M) and args[1].dtype == torch.float32:
        with pytest.raises(exc, match="must"):
            w.f8_gemm_gated(*args[:2], *more, *args[2:])


def test_gated_options(cpu_ok):
    args = (f8(M, K), f32(KB, M), f8(N, K), f32(NB, KB), f8(N, K), f32(NB, KB))
    with pytest.raises(ValueError, match="activation"):
        w.f8_gemm_gated(*args, "relu")
    with pytest.raises(ValueError):
        w.f8_gemm_gated(*args, 7)
    with pytest.raises(TypeError, match="out must be"):
        w.f8_gemm_gated(*args, out=f16(M, N))
    with pytest.raises(ValueError, match="scale must be"):
        w.f8_gemm_gated(*args, scale=f32(M, NB))
    with pytest.raises(ValueError, match="scale must be None"):
        w.f8_gemm_gated(*args, quantize=False, scale=f32(NB, M))


def test_norm_operands(cpu_ok):
    x, g = f16(M, 256), f16(256)
    with pytest.raises(ValueError, match="gain must"):
        w.rmsnorm_quant(w.Mode.F8, x, f16(255))
    with pytest.raises(TypeError, match="gain must"):
        w.rmsnorm_quant(w.Mode.F8, x, g.float())
    with pytest.raises(TypeError, match="x must"):
        w.rmsnorm_quant(w.Mode.F8, x.float(), g)
    with pytest.raises(ValueError, match="residual must"):
        w.rmsnorm_quant(w.Mode.F8, x, g, residual=f16(M + 1, 256))
    with pytest.raises(ValueError, match="residual_out must be None"):
        w.rmsnorm_quant(w.Mode.F8, x, g, residual_out=f16(M, 256))
    with pytest.raises(ValueError, match="residual_out must"):
        w.rmsnorm_quant(w.Mode.F8, x, g, residual=x, residual_out=f16(M, 128))
    with pytest.raises(ValueError, match="group_size"):
        w.rmsnorm_quant(w.Mode.W8A8_PG, x, g)
    with pytest.raises(ValueError, match="scale must"):
        w.rmsnorm_quant(w.Mode.W8A8_PC, x, g, scale=f32(M, 1))
    with pytest.raises(TypeError, match="out must"):
        w.rmsnorm_quant(w.Mode.F8, x, g, out=torch.zeros(M, 256, dtype=torch.int8))
    with pytest.raises(ValueError):
        w.rmsnorm_quant(9, x, g)


def test_linear_operands(cpu_ok):
    with pytest.raises(ValueError, match="w_scale must"):
        w.linear(w.Mode.F8, f16(M, K), f8(N, K), f32(N))
    with pytest.raises(TypeError, match="w must"):
        w.linear(w.Mode.F8, f16(M, K), torch.zeros(N, K, dtype=torch.int8), f32(NB, KB))
    need = w.linear_workspace_size(w.Mode.F8, M, K)
    assert need >= M * K + KB * M * 4
    with pytest.raises(ValueError, match="workspace"):
        w.linear(w.Mode.F8, f16(M, K), f8(N, K), f32(NB, KB), workspace=torch.zeros(need - 1, dtype=torch.uint8))


def test_sizes():
    assert w.linear_workspace_size(w.Mode.F8, 0, 256) == 0
    assert w.linear_workspace_size(w.Mode.F8, 1, 256) > 0
    for size in (w.f8_gemm_workspace_size, w.f8_gemm_gated_workspace_size):
        assert size(0, 128, 128) == 0 and size(-3, 128, 128) == 0 and size(4, 128, -1) == 0
