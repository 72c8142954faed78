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
import functools

import torch

from . import ops
from ._lib import CacheStruct, check, lib
from .ops import _need, _shaped

# A decode step calls these for microseconds of GPU work each, so the checks are
# kept short: pointers go to ctypes as integers, the stream is torch's current
# one as a number, and the device is only switched when it is not the current.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(index):
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def _call(index, fn, *args):
    """fn(*args, stream) with device `index` current."""
    if torch.cuda.current_device() == index:
        status = fn(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _stream(index))
    if status:
        check(status)


_LARGEST = 2 ** 31 - 1


def _at_most(n, most):
    """n cut to [-1, most]: ctypes would take a longer number modulo 2^32."""
    return -1 if n < 0 else n if n < most else most


def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _rows(t, name, index=None, heads=None, head_dim=None):
    """fp16 [T, heads, head_dim] whose heads are contiguous in a token; tokens may be strided.
    Returns (T, elements from one token to the next)."""
    if not isinstance(t, torch.Tensor):
        _tensor(t, name)
    if index is None:
        if t.device.type != ops._DEVICE_TYPE:
            raise ValueError(f"{name} must be a device tensor, got {t.device}")
    elif t.get_device() != index:
        raise ValueError(f"{name} must be on the device of the other operands, got {t.device}")
    if t.dtype is not torch.float16:
        raise TypeError(f"{name} must be torch.float16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims [T, heads, head_dim], got shape {tuple(t.shape)}")
    T, h, d = t.shape
    if (heads is not None and h != heads) or (head_dim is not None and d != head_dim):
        raise ValueError(f"{name} must have shape [T, {heads}, {head_dim}], got {tuple(t.shape)}")
    st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError(f"{name} must have contiguous heads within a token, got strides {(st, sh, sd)}")
    return T, st if T > 1 else h * d


def _flat(t, dtype, shape, name, index):
    """t must be a contiguous `dtype` tensor of exactly `shape` on device `index`."""
    if not isinstance(t, torch.Tensor):
        _tensor(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got shape {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the device of the other operands, got {t.device}")
    return t


class KV4Cache:
    """A paged key/value cache in 4 bits over four tensors that the caller owns:

    k, v              uint8 [pages, kv_heads, page_size, head_dim / 2]
    k_scale, v_scale  fp32  [pages, kv_heads, page_size, head_dim / group_size]

    Slot s is row s % page_size of page s // page_size.  The tensors are checked
    once here; the object keeps them and the C description of them.
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "pages", "kv_heads", "page_size", "head_dim",
                 "group_size", "device", "_index", "_struct", "_ref")

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
        self.device, self._index = k.device, k.get_device()
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


@functools.lru_cache(maxsize=64)
def _sections(sections, half):
    """The C array of an axis' pair counts, checked."""
    if not 1 <= len(sections) <= 3 or min(sections) < 0 or sum(sections) != half:
        raise ValueError(f"sections must be 1 to 3 counts that sum to {half}, got {sections}")
    return (ctypes.c_int32 * len(sections))(*sections)


def rotary_axes(x, positions, inv_freq, sections=None, interleaved: bool = False, out=None):
    """Rotary positions: x fp16 [T, heads, head_dim] (tokens may be strided), positions int64
    [axes, T] (or [T]), inv_freq fp32 [rotary_dim / 2]; sections: how many pairs each axis
    turns (default: one axis turns all).  out (default: a new tensor) may be x."""
    T, stride = _rows(x, "x")
    _, heads, D = x.shape
    index = x.get_device()
    if not isinstance(inv_freq, torch.Tensor) or not isinstance(positions, torch.Tensor):
        _tensor(inv_freq, "inv_freq")
        _tensor(positions, "positions")
    half = inv_freq.numel()
    _flat(inv_freq, torch.float32, (half,), "inv_freq", index)
    if half == 0 or half % 8 or 2 * half > D:
        raise ValueError(f"inv_freq must have rotary_dim / 2 values, a multiple of 8 up to {D // 2}, "
                         f"got {half}")
    counts = _sections((half,) if sections is None else tuple(sections), half)
    axes = len(counts)
    flat = positions.dim() == 1 and axes == 1
    _flat(positions, torch.int64, (T,) if flat else (axes, T), "positions", index)
    if out is None:
        out = torch.empty((T, heads, D), dtype=torch.float16, device=x.device)
        out_stride = heads * D
    elif _rows(out, "out", index, heads, D)[0] != T:
        raise ValueError(f"out must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
    else:
        out_stride = _rows(out, "out", index, heads, D)[1]
    _call(index, lib().rotary_axes, x.data_ptr(), stride, positions.data_ptr(), inv_freq.data_ptr(), T, heads, D,
          2 * half, axes, counts, interleaved, out.data_ptr(), out_stride)
    return out


def kv4_write(k, v, slots, cache):
    """Quantize T tokens' keys and values (fp16 [T, kv_heads, head_dim], tokens may be strided)
    into the cache's slots (int64 [T]; outside the cache: not written)."""
    index = _cache(cache)._index
    T, k_stride = _rows(k, "k", index, cache.kv_heads, cache.head_dim)
    Tv, v_stride = _rows(v, "v", index, cache.kv_heads, cache.head_dim)
    if Tv != T:
        raise ValueError(f"v has {Tv} tokens, k has {T}: shape mismatch")
    _flat(slots, torch.int64, (T,), "slots", index)
    _call(index, lib().kv4_write, k.data_ptr(), k_stride, v.data_ptr(), v_stride, slots.data_ptr(), T, cache._ref)


def kv4_read(cache, slots, k=None, v=None):
    """The keys and values of T slots (int64 [T]) as fp16 [T, kv_heads, head_dim] each."""
    index = _cache(cache)._index
    T = _tensor(slots, "slots").numel()
    _flat(slots, torch.int64, (T,), "slots", index)
    shape = (T, cache.kv_heads, cache.head_dim)
    if k is None:
        k = torch.empty(shape, dtype=torch.float16, device=cache.device)
    else:
        _flat(k, torch.float16, shape, "k", index)
    if v is None:
        v = torch.empty(shape, dtype=torch.float16, device=cache.device)
    else:
        _flat(v, torch.float16, shape, "v", index)
    _call(index, lib().kv4_read, cache._ref, slots.data_ptr(), T, k.data_ptr(), v.data_ptr())
    return k, v


def kv4_attention_workspace_size(q_heads: int, kv_heads: int, head_dim: int, tokens: int,
                                 sequences: int, max_q: int = 1) -> int:
    return int(lib().kv4_attention_workspace_size(q_heads, kv_heads, head_dim, tokens, sequences,
                                                  _at_most(max_q, tokens)))


def kv4_attention_workspace(cache, q_heads: int, tokens: int, sequences: int, max_q: int = 1):
    """A workspace for calls of kv4_attention of these sizes, to be kept between calls that do not
    overlap."""
    _cache(cache)
    need = kv4_attention_workspace_size(q_heads, cache.kv_heads, cache.head_dim, tokens, sequences,
                                        max_q)
    return torch.empty((need,), dtype=torch.uint8, device=cache.device)


def kv4_attention(q, cache, page_table, kv_lens, q_starts=None, max_q=None, causal: bool = True,
                  window: int = 0, scale=None, workspace=None, out=None, lse=None,
                  return_lse: bool = False):
    """Attention of T query rows (fp16 [T, q_heads, head_dim], tokens may be strided) over the
    cache: page_table int32 [sequences, max_pages], kv_lens int32 [sequences] (the queries' own
    tokens counted), q_starts int32 [sequences + 1] (default: one query a sequence), max_q an
    upper bound of a sequence's queries (default: T with q_starts, which suits any; rows past it
    and rows in no sequence are not written).  scale defaults to head_dim ** -0.5.  workspace: of
    kv4_attention_workspace (default: a new one).  Returns out fp16 [T, q_heads, head_dim], with
    return_lse (out, lse fp32 [T, q_heads])."""
    index = _cache(cache)._index
    T, stride = _rows(q, "q", index)
    _, heads, D = q.shape
    if D != cache.head_dim or heads == 0 or heads % cache.kv_heads:
        raise ValueError(f"q must have head_dim {cache.head_dim} and a multiple of {cache.kv_heads} "
                         f"heads, got shape {tuple(q.shape)}")
    if _tensor(page_table, "page_table").dim() != 2:
        raise ValueError(f"page_table must have 2 dims, got shape {tuple(page_table.shape)}")
    B, max_pages = page_table.shape
    _flat(page_table, torch.int32, (B, max_pages), "page_table", index)
    _flat(kv_lens, torch.int32, (B,), "kv_lens", index)
    if q_starts is not None:
        starts = _flat(q_starts, torch.int32, (B + 1,), "q_starts", index).data_ptr()
    elif T != B:
        raise ValueError(f"without q_starts q must have one row a sequence, got shape {tuple(q.shape)} "
                         f"for {B} sequences")
    else:
        starts = None
    if max_q is None:
        max_q = 1 if q_starts is None else T
    max_q = _at_most(max_q, T)
    L = lib()
    if workspace is None:
        need = L.kv4_attention_workspace_size(heads, cache.kv_heads, D, T, B, max_q)
        workspace = torch.empty((need,), dtype=torch.uint8, device=cache.device)
    else:
        _flat(workspace, torch.uint8, (_tensor(workspace, "workspace").numel(),), "workspace", index)     # its size: by the library
    shape = (T, heads, D)
    if out is None:
        out = torch.empty(shape, dtype=torch.float16, device=cache.device)
    else:
        _flat(out, torch.float16, shape, "out", index)
    if lse is not None:
        _flat(lse, torch.float32, (T, heads), "lse", index)
    elif return_lse:
        lse = torch.empty((T, heads), dtype=torch.float32, device=cache.device)
    _call(index, L.kv4_attention, q.data_ptr(), stride, T, heads, cache._ref, page_table.data_ptr(), max_pages,
          kv_lens.data_ptr(), starts, B, max_q, causal, _at_most(window, _LARGEST), D ** -0.5 if scale is None else scale,
          out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return (out, lse) if return_lse else out
