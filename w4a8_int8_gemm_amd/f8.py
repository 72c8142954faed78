"""The wrappers of 8-bit floating point in blocks of 128 and of the norm in
front of the linear layers (marshalling only, as in ops.py).

    q, s, h = rmsnorm_quant(Mode.F8, x, gain, 1e-6, residual=h)       # h = x + h, its norm in 8 bits
    a, a_s = f8_gemm_gated(q, s, wg, wg_s, wu, wu_s, "silu")          # again in 8 bits
    y = f8_gemm(a, a_s, wd, wd_s)                                     # fp16 [M, N]
    y = linear(Mode.F8, x, w, w_scale)                                # from fp16 activations

Codes are torch.float8_e4m3fn; activations' scales are fp32 [ceil(K / 128), M]
(the tokens side by side), weights' fp32 [ceil(N / 128), ceil(K / 128)].
"""
from __future__ import annotations

import torch

from . import ops
from ._lib import Activation, Mode, lib
from .kv4 import _flat, _tensor
from .ops import _call, _need, _out

F8, F16, F32 = torch.float8_e4m3fn, torch.float16, torch.float32
_ACTIVATIONS = {"silu": Activation.SILU, "gelu_tanh": Activation.GELU_TANH}
_empty, _empty_like = torch.empty, torch.empty_like


def _blocks(n):
    return (n + 127) // 128


def _matrix(t, dtype, name):
    """A contiguous `dtype` matrix on a device: its rows, columns and device index."""
    if not isinstance(t, torch.Tensor):
        _tensor(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous matrix, got shape {tuple(t.shape)} and strides {t.stride()}")
    if t.device.type != ops._DEVICE_TYPE:
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    rows, columns = t.shape
    return rows, columns, t.get_device()


def quantize_act_f8(x, out=None, scale=None):
    """fp16 [M, K] -> (e4m3 [M, K], fp32 [ceil(K / 128), M])."""
    M, K, index = _matrix(x, F16, "x")
    out = _empty_like(x, dtype=F8) if out is None else _flat(out, F8, (M, K), "out", index)
    shape = (_blocks(K), M)
    scale = _empty(shape, dtype=F32, device=x.device) if scale is None else _flat(scale, F32, shape, "scale", index)
    _call(index, lib().quantize_act_f8, x.data_ptr(), M, K, out.data_ptr(), scale.data_ptr())
    return out, scale


def quantize_weight_f8(w, out=None, scale=None):
    """fp16 [N, K] -> (e4m3 [N, K], fp32 [ceil(N / 128), ceil(K / 128)])."""
    _need(w, torch.float16, "w", 2)
    N, K = w.shape
    out = _out(out, (N, K), F8, w, "out")
    scale = _out(scale, (_blocks(N), _blocks(K)), torch.float32, w, "scale")
    _call(w.get_device(), lib().quantize_weight_f8, w.data_ptr(), N, K, out.data_ptr(), scale.data_ptr())
    return out, scale


def rmsnorm_quant(mode, x, gain, eps: float = 1e-6, residual=None, group_size: int = 0, out=None,
                  scale=None, residual_out=None):
    """h = x + residual; the root-mean-square norm of h times gain, quantized as linear layers of
    `mode` take their activations: int8 with fp32 scales [M] (W8A8_PC, W4A8) or [M, K / group_size]
    (W8A8_PG), or e4m3 with fp32 scales [ceil(K / 128), M] (F8).  x, residual fp16 [M, K], gain
    fp16 [K].  Returns (codes, scales), with a residual (codes, scales, fp16(h)); residual_out may
    be residual or x."""
    if mode.__class__ is not Mode:
        mode = Mode(mode)
    M, K, index = _matrix(x, F16, "x")
    _flat(gain, F16, (K,), "gain", index)
    if mode is Mode.F8:
        dtype, shape, group_size = F8, (_blocks(K), M), 0
    elif mode is Mode.W8A8_PG:
        dtype, shape = torch.int8, (M, ops._groups(K, group_size))
    else:
        dtype, shape, group_size = torch.int8, (M,), 0
    out = _empty_like(x, dtype=dtype) if out is None else _flat(out, dtype, (M, K), "out", index)
    scale = _empty(shape, dtype=F32, device=x.device) if scale is None else _flat(scale, F32, shape, "scale", index)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out must be None without a residual")
        _call(index, lib().rmsnorm_quant, mode, x.data_ptr(), None, gain.data_ptr(), eps, M, K, group_size,
              out.data_ptr(), scale.data_ptr(), None)
        return out, scale
    _flat(residual, F16, (M, K), "residual", index)
    residual_out = _empty_like(x) if residual_out is None else _flat(residual_out, F16, (M, K), "residual_out", index)
    _call(index, lib().rmsnorm_quant, mode, x.data_ptr(), residual.data_ptr(), gain.data_ptr(), eps, M, K, group_size,
          out.data_ptr(), scale.data_ptr(), residual_out.data_ptr())
    return out, scale, residual_out


def _workspace(workspace, need, index, device):
    """(the workspace, a new one where none is given, to be kept until the call is made; its address; bytes)."""
    if workspace is None:
        workspace = _empty((need,), dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    size = _tensor(workspace, "workspace").numel()
    _flat(workspace, torch.uint8, (size,), "workspace", index)     # its size: by the library
    return workspace, workspace.data_ptr(), size


def f8_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().f8_gemm_workspace_size(M, N, K))


def f8_gemm_workspace(M: int, N: int, K: int, device="cuda"):
    """A workspace for calls of f8_gemm of these sizes, to be kept between calls that do not overlap."""
    return torch.empty((f8_gemm_workspace_size(M, N, K),), dtype=torch.uint8, device=device)


def _weights(w, scale, N, K, name, index):
    _flat(w, F8, (N, K), name, index)
    _flat(scale, F32, (_blocks(N), _blocks(K)), name + "_scale", index)


def _rows_of(w, name):
    if _tensor(w, name).dim() != 2:
        raise ValueError(f"{name} must be a contiguous matrix, got shape {tuple(w.shape)}")
    return w.shape[0]


def f8_gemm(xq, x_scale, w, w_scale, out=None, workspace=None):
    """y fp16 [M, N] = xq . w^T with their blocks' scales: xq e4m3 [M, K], x_scale fp32
    [ceil(K / 128), M], w e4m3 [N, K], w_scale fp32 [ceil(N / 128), ceil(K / 128)].  workspace: of
    f8_gemm_workspace (default: a new one)."""
    M, K, index = _matrix(xq, F8, "xq")
    _flat(x_scale, F32, (_blocks(K), M), "x_scale", index)
    N = _rows_of(w, "w")
    _weights(w, w_scale, N, K, "w", index)
    out = _empty((M, N), dtype=F16, device=xq.device) if out is None else _flat(out, F16, (M, N), "out", index)
    L = lib()
    need = L.f8_gemm_workspace_size(M, N, K)
    if need or workspace is not None:
        workspace, at, size = _workspace(workspace, need, index, xq.device)
    else:
        at, size = None, 0
    _call(index, L.f8_gemm, xq.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), out.data_ptr(),
          M, N, K, at, size)
    return out


def f8_gemm_gated_workspace_size(M: int, N: int, K: int, quantize: bool = True) -> int:
    return int(lib().f8_gemm_gated_workspace_size(M, N, K, bool(quantize)))


def f8_gemm_gated_workspace(M: int, N: int, K: int, quantize: bool = True, device="cuda"):
    """A workspace for calls of f8_gemm_gated of these sizes, to be kept between calls that do not overlap."""
    return torch.empty((f8_gemm_gated_workspace_size(M, N, K, quantize),), dtype=torch.uint8, device=device)


def f8_gemm_gated(xq, x_scale, w_gate, gate_scale, w_up, up_scale, activation="silu", quantize: bool = True,
                  out=None, scale=None, workspace=None):
    """act(xq . w_gate^T) * (xq . w_up^T), the first half of a gated feed-forward block: operands as
    f8_gemm's, activation "silu" or "gelu_tanh" (or an Activation).  With quantize (e4m3 [M, N],
    fp32 [ceil(N / 128), M]), ready for f8_gemm; without, fp16 [M, N]."""
    M, K, index = _matrix(xq, F8, "xq")
    _flat(x_scale, F32, (_blocks(K), M), "x_scale", index)
    N = _rows_of(w_gate, "w_gate")
    _weights(w_gate, gate_scale, N, K, "w_gate", index)
    _weights(w_up, up_scale, N, K, "w_up", index)
    act = _ACTIVATIONS.get(activation) if isinstance(activation, str) else Activation(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, got {activation!r}")
    dtype = F8 if quantize else F16
    out = _empty((M, N), dtype=dtype, device=xq.device) if out is None else _flat(out, dtype, (M, N), "out", index)
    if quantize:
        shape = (_blocks(N), M)
        scale = _empty(shape, dtype=F32, device=xq.device) if scale is None else _flat(scale, F32, shape, "scale", index)
    elif scale is not None:
        raise ValueError("scale must be None without quantize")
    L = lib()
    need = L.f8_gemm_gated_workspace_size(M, N, K, bool(quantize))
    if need or workspace is not None:
        workspace, at, size = _workspace(workspace, need, index, xq.device)
    else:
        at, size = None, 0
    y, yq, ys = (None, out.data_ptr(), scale.data_ptr()) if quantize else (out.data_ptr(), None, None)
    _call(index, L.f8_gemm_gated, xq.data_ptr(), x_scale.data_ptr(), w_gate.data_ptr(), gate_scale.data_ptr(),
          w_up.data_ptr(), up_scale.data_ptr(), act, M, N, K, y, yq, ys, at, size)
    return (out, scale) if quantize else out
