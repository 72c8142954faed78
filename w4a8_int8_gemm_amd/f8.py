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
from .kv4 import _call, _flat, _tensor
from .ops import _need, _out

F8 = torch.float8_e4m3fn
_ACTIVATIONS = {"silu": Activation.SILU, "gelu_tanh": Activation.GELU_TANH}


def _blocks(n):
    return (n + 127) // 128


def _matrix(t, dtype, name, index=None):
    """A contiguous `dtype` matrix on a device (device `index`): its shape."""
    if not isinstance(t, torch.Tensor):
        _tensor(t, name)
    if index is None:
        if t.device.type != ops._DEVICE_TYPE:
            raise ValueError(f"{name} must be a device tensor, got {t.device}")
    elif t.get_device() != index:
        raise ValueError(f"{name} must be on the device of the other operands, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous matrix, got shape {tuple(t.shape)} and strides {t.stride()}")
    return t.shape


def _give(t, dtype, shape, name, index, device):
    """The output t, checked, or a new one."""
    return torch.empty(shape, dtype=dtype, device=device) if t is None else _flat(t, dtype, shape, name, index)


def quantize_act_f8(x, out=None, scale=None):
    """fp16 [M, K] -> (e4m3 [M, K], fp32 [ceil(K / 128), M])."""
    M, K = _matrix(x, torch.float16, "x")
    index = x.get_device()
    out = _give(out, F8, (M, K), "out", index, x.device)
    scale = _give(scale, torch.float32, (_blocks(K), M), "scale", index, x.device)
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
    mode = Mode(mode)
    M, K = _matrix(x, torch.float16, "x")
    index = x.get_device()
    _flat(gain, torch.float16, (K,), "gain", index)
    if mode == Mode.F8:
        dtype, shape = F8, (_blocks(K), M)
    elif mode == Mode.W8A8_PG:
        dtype, shape = torch.int8, (M, ops._groups(K, group_size))
    else:
        dtype, shape = torch.int8, (M,)
    if residual is not None:
        _flat(residual, torch.float16, (M, K), "residual", index)
        residual_out = _give(residual_out, torch.float16, (M, K), "residual_out", index, x.device)
    elif residual_out is not None:
        raise ValueError("residual_out must be None without a residual")
    out = _give(out, dtype, (M, K), "out", index, x.device)
    scale = _give(scale, torch.float32, shape, "scale", index, x.device)
    _call(index, lib().rmsnorm_quant, int(mode), x.data_ptr(), None if residual is None else residual.data_ptr(),
          gain.data_ptr(), eps, M, K, group_size if mode == Mode.W8A8_PG else 0, out.data_ptr(), scale.data_ptr(),
          None if residual is None else residual_out.data_ptr())
    return (out, scale) if residual is None else (out, scale, residual_out)


def _workspace(workspace, need, index, device):
    """(address, bytes) of the workspace, a new one where none is given; it is returned too, to be kept until
    the call is made."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty((need,), dtype=torch.uint8, device=device)
    else:
        _flat(workspace, torch.uint8, (_tensor(workspace, "workspace").numel(),), "workspace", index)  # its size: by the library
    return workspace, workspace.data_ptr(), workspace.numel()


def f8_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().f8_gemm_workspace_size(M, N, K))


def f8_gemm_workspace(M: int, N: int, K: int, device="cuda"):
    """A workspace for calls of f8_gemm of these sizes, to be kept between calls that do not overlap."""
    return torch.empty((f8_gemm_workspace_size(M, N, K),), dtype=torch.uint8, device=device)


def _weights(w, scale, N, K, name, index):
    _flat(w, F8, (N, K), name, index)
    _flat(scale, torch.float32, (_blocks(N), _blocks(K)), name + "_scale", index)


def _codes(xq, x_scale):
    M, K = _matrix(xq, F8, "xq")
    index = xq.get_device()
    _flat(x_scale, torch.float32, (_blocks(K), M), "x_scale", index)
    return M, K, index


def f8_gemm(xq, x_scale, w, w_scale, out=None, workspace=None):
    """y fp16 [M, N] = xq . w^T with their blocks' scales: xq e4m3 [M, K], x_scale fp32
    [ceil(K / 128), M], w e4m3 [N, K], w_scale fp32 [ceil(N / 128), ceil(K / 128)].  workspace: of
    f8_gemm_workspace (default: a new one)."""
    M, K, index = _codes(xq, x_scale)
    N = _matrix(w, F8, "w", index)[0]
    _weights(w, w_scale, N, K, "w", index)
    out = _give(out, torch.float16, (M, N), "out", index, xq.device)
    L = lib()
    keep, at, size = _workspace(workspace, L.f8_gemm_workspace_size(M, N, K), index, xq.device)
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
    M, K, index = _codes(xq, x_scale)
    N = _matrix(w_gate, F8, "w_gate", index)[0]
    _weights(w_gate, gate_scale, N, K, "w_gate", index)
    _weights(w_up, up_scale, N, K, "w_up", index)
    act = _ACTIVATIONS.get(activation) if isinstance(activation, str) else Activation(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, got {activation!r}")
    if not quantize and scale is not None:
        raise ValueError("scale must be None without quantize")
    out = _give(out, F8 if quantize else torch.float16, (M, N), "out", index, xq.device)
    if quantize:
        scale = _give(scale, torch.float32, (_blocks(N), M), "scale", index, xq.device)
    L = lib()
    keep, at, size = _workspace(workspace, L.f8_gemm_gated_workspace_size(M, N, K, bool(quantize)), index, xq.device)
    _call(index, L.f8_gemm_gated, xq.data_ptr(), x_scale.data_ptr(), w_gate.data_ptr(), gate_scale.data_ptr(),
          w_up.data_ptr(), up_scale.data_ptr(), int(act), M, N, K, None if quantize else out.data_ptr(),
          out.data_ptr() if quantize else None, scale.data_ptr() if quantize else None, at, size)
    return (out, scale) if quantize else out
