"""The attention block's wrappers: rotary positions, the 4-bit paged key/value
cache and attention over it (marshalling only, as in ops.py).

    x = linear(Mode.W4A8, h, w4, sw, 128).view(T, q_heads + 2 * kv_heads, head_dim)
    qk = rotary_axes(x[:, :q_heads + kv_heads], positions, inv_freq, (24, 20, 20), interleaved=True)
    cache = KV4Cache.empty(pages, kv_heads, page_size=64, head_dim=128, group_size=64)
    kv4_write(qk[:, q_heads:], x[:, q_heads + kv_heads:], slots, cache)
    o = kv4_attention(qk[:, :q_heads], cache, page_table, kv_lens, q_starts=q_starts, max_q=max_q)
"""
from __future__ import annotations

import ctypes

import torch

from . import ops
from ._lib import CacheStruct, check, lib
from .ops import _need, _out, _p, _shaped, _st


def _rows(t, name, like=None, heads=None, head_dim=None):
    """fp16 [T, heads, head_dim] whose heads are contiguous in a token; tokens may be strided."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != ops._DEVICE_TYPE:
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {like.device}")
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be torch.float16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims [T, heads, head_dim], got shape {tuple(t.shape)}")
    T, h, d = t.shape
    if (heads is not None and h != heads) or (head_dim is not None and d != head_dim):
        raise ValueError(f"{name} must have shape [T, {heads}, {head_dim}], got {tuple(t.shape)}")
    st = t.stride()
    if (d > 1 and st[2] != 1) or (h > 1 and st[1] != d):
        raise ValueError(f"{name} must have contiguous heads within a token, got strides {st}")
    return t


def _token_stride(t):
    """Elements from one token to the next (a single token has none of its own)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


class KV4Cache:
    """A paged key/value cache in 4 bits over four tensors that the caller owns:

    k, v              uint8 [pages, kv_heads, page_size, head_dim / 2]
    k_scale, v_scale  fp32  [pages, kv_heads, page_size, head_dim / group_size]

    Slot s is row s % page_size of page s // page_size.  The tensors are checked
    once here; the object keeps them and the C description of them.
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "pages", "kv_heads", "page_size", "head_dim",
                 "group_size", "device", "_struct", "_ref")

    def __init__(self, k, k_scale, v, v_scale):
        _need(k, torch.uint8, "k", 4)
        pages, heads, page, half = k.shape
        _need(k_scale, torch.float32, "k_scale", 4, k)
        groups = k_scale.shape[3]
        if groups == 0 or (2 * half) % groups:
            raise ValueError(f"k_scale has {groups} groups for head_dim {2 * half}")
        _shaped(k_scale, torch.float32, (pages, heads, page, groups), "k_scale", k)
        _shaped(v, torch.uint8, (pages, heads, page, half), "v", k)
        _shaped(v_scale, torch.float32, (pages, heads, page, groups), "v_scale", k)
        if 2 * half not in (64, 128, 256):
            raise ValueError(f"head_dim must be 64, 128 or 256, got {2 * half}")
        if groups not in (1, 2, 4) or 2 * half // groups < 32:
            raise ValueError("group_size must be 32, 64, 128 or 256, at most head_dim and at least a "
                             f"quarter of it, got {2 * half // groups} for head_dim {2 * half}")
        if page < 16 or page > 1 << 20 or page & (page - 1):
            raise ValueError(f"page_size must be a power of two in [16, 2^20], got {page}")
        if pages < 1 or heads < 1:
            raise ValueError(f"the cache must have pages and heads, got shape {tuple(k.shape)}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.kv_heads, self.page_size = pages, heads, page
        self.head_dim, self.group_size = 2 * half, 2 * half // groups
        self.device = k.device
        self._struct = CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                   pages, heads, page, self.head_dim, self.group_size)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page_size: int = 64, head_dim: int = 128,
              group_size: int = 64, device="cuda"):
        """A cache of uninitialised pages."""
        if group_size <= 0 or head_dim % group_size:
            raise ValueError(f"group_size={group_size} does not divide head_dim={head_dim}")

        def make(n, dtype):
            return torch.empty((pages, kv_heads, page_size, n), dtype=dtype, device=device)

        return cls(make(head_dim // 2, torch.uint8), make(head_dim // group_size, torch.float32),
                   make(head_dim // 2, torch.uint8), make(head_dim // group_size, torch.float32))


def _cache(c):
    if not isinstance(c, KV4Cache):
        raise TypeError("cache must be a KV4Cache")
    return c


def rotary_axes(x, positions, inv_freq, sections=None, interleaved: bool = False, out=None):
    """Rotary positions: x fp16 [T, heads, head_dim] (tokens may be strided), positions int64
    [axes, T] (or [T]), inv_freq fp32 [rotary_dim / 2]; sections: how many pairs each axis
    turns (default: one axis turns all).  out (default: a new tensor) may be x."""
    _rows(x, "x")
    T, heads, D = x.shape
    _need(inv_freq, torch.float32, "inv_freq", 1, x)
    half = inv_freq.shape[0]
    if half == 0 or half % 8 or 2 * half > D:
        raise ValueError(f"inv_freq must have rotary_dim / 2 values, a multiple of 8 up to {D // 2}, "
                         f"got {half}")
    sections = (half,) if sections is None else tuple(int(n) for n in sections)
    axes = len(sections)
    if not 1 <= axes <= 3 or min(sections) < 0 or sum(sections) != half:
        raise ValueError(f"sections must be 1 to 3 counts that sum to {half}, got {sections}")
    if positions.dim() == 1:
        positions = positions.unsqueeze(0)
    _shaped(positions, torch.int64, (axes, T), "positions", x)
    if out is None:
        out = torch.empty((T, heads, D), dtype=torch.float16, device=x.device)
    else:
        _rows(out, "out", x, heads, D)
        if out.shape[0] != T:
            raise ValueError(f"out must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
    with torch.cuda.device(x.device):
        check(lib().rotary_axes(_p(x), _token_stride(x), _p(positions), _p(inv_freq), T, heads, D,
                                2 * half, axes, (ctypes.c_int32 * axes)(*sections),
                                int(interleaved), _p(out), _token_stride(out), _st(x)))
    return out


def kv4_write(k, v, slots, cache):
    """Quantize T tokens' keys and values (fp16 [T, kv_heads, head_dim], tokens may be strided)
    into the cache's slots (int64 [T]; outside the cache: not written)."""
    _cache(cache)
    _rows(k, "k", cache, cache.kv_heads, cache.head_dim)
    _rows(v, "v", cache, cache.kv_heads, cache.head_dim)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError(f"v has {v.shape[0]} tokens, k has {T}: shape mismatch")
    _shaped(slots, torch.int64, (T,), "slots", cache)
    with torch.cuda.device(cache.device):
        check(lib().kv4_write(_p(k), _token_stride(k), _p(v), _token_stride(v), _p(slots), T,
                              cache._ref, _st(k)))


def kv4_read(cache, slots, k=None, v=None):
    """The keys and values of T slots (int64 [T]) as fp16 [T, kv_heads, head_dim] each."""
    _cache(cache)
    _need(slots, torch.int64, "slots", 1, cache)
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    k = _out(k, shape, torch.float16, cache, "k")
    v = _out(v, shape, torch.float16, cache, "v")
    with torch.cuda.device(cache.device):
        check(lib().kv4_read(cache._ref, _p(slots), shape[0], _p(k), _p(v), _st(slots)))
    return k, v


def kv4_attention_workspace_size(q_heads: int, kv_heads: int, head_dim: int, tokens: int,
                                 sequences: int, max_q: int = 1) -> int:
    return int(lib().kv4_attention_workspace_size(q_heads, kv_heads, head_dim, tokens, sequences,
                                                  max_q))


def kv4_attention_workspace(cache, q_heads: int, tokens: int, sequences: int, max_q: int = 1):
    """A workspace for calls of kv4_attention up to these sizes, to be kept between calls that do
    not overlap."""
    _cache(cache)
    need = kv4_attention_workspace_size(q_heads, cache.kv_heads, cache.head_dim, tokens, sequences,
                                        max_q)
    return torch.empty((need,), dtype=torch.uint8, device=cache.device)


def kv4_attention(q, cache, page_table, kv_lens, q_starts=None, max_q: int = 1, causal: bool = True,
                  window: int = 0, scale=None, workspace=None, out=None, lse=None,
                  return_lse: bool = False):
    """Attention of T query rows (fp16 [T, q_heads, head_dim], tokens may be strided) over the
    cache: page_table int32 [sequences, max_pages], kv_lens int32 [sequences] (the queries' own
    tokens counted), q_starts int32 [sequences + 1] (default: one query a sequence), max_q an
    upper bound of a sequence's queries.  scale defaults to head_dim ** -0.5.  Returns out fp16
    [T, q_heads, head_dim], with return_lse (out, lse fp32 [T, q_heads])."""
    _cache(cache)
    _rows(q, "q", cache, None, None)
    T, heads, D = q.shape
    if D != cache.head_dim or heads == 0 or heads % cache.kv_heads:
        raise ValueError(f"q must have head_dim {cache.head_dim} and a multiple of {cache.kv_heads} "
                         f"heads, got shape {tuple(q.shape)}")
    _need(page_table, torch.int32, "page_table", 2, cache)
    B, max_pages = page_table.shape
    _shaped(kv_lens, torch.int32, (B,), "kv_lens", cache)
    if q_starts is not None:
        _shaped(q_starts, torch.int32, (B + 1,), "q_starts", cache)
    elif T != B:
        raise ValueError(f"without q_starts q must have one row a sequence, got shape {tuple(q.shape)} "
                         f"for {B} sequences")
    need = lib().kv4_attention_workspace_size(heads, cache.kv_heads, D, T, B, max_q)
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=cache.device)
    else:
        _need(workspace, torch.uint8, "workspace", 1, cache)
        if workspace.numel() < need:
            raise ValueError(f"workspace has {workspace.numel()} bytes, {need} needed")
    out = _out(out, (T, heads, D), torch.float16, cache, "out")
    if return_lse or lse is not None:
        lse = _out(lse, (T, heads), torch.float32, cache, "lse")
    with torch.cuda.device(cache.device):
        check(lib().kv4_attention(_p(q), _token_stride(q), T, heads, cache._ref, _p(page_table),
                                  max_pages, _p(kv_lens), _p(q_starts), B, max_q, int(causal),
                                  window, D ** -0.5 if scale is None else scale, _p(out), _p(lse),
                                  _p(workspace), workspace.numel(), _st(q)))
    return (out, lse) if return_lse else out
