"""Binding of the 4-bit paged KV cache (kv4_* of include/moe_verify.h).

Thin like ``api``: argument checks and pointer marshalling; tensors are on one
CUDA device, calls enqueue on the current stream (or ``stream``) and raise
``MoEError`` on a non-OK host status.  Device-side error bits land in
``dev_err`` where one is given.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Tuple

import torch

from . import _lib as L
from .api import MoEError, _check, _need, _ptr, _stream

_DTYPES = {torch.float32: L.DTYPE_F32, torch.bfloat16: L.DTYPE_BF16}


class Kv4Cache:
    """Pages and page table of a batch's cache.

    ``pages`` uint8 [n_pages, n_kv_heads, page_size * (head_dim + 8)] and ``table`` int32 [n_seq, max_pages]
    stay the caller's: the table's contents (which page holds a sequence's slots) may change between calls.
    """

    def __init__(self, pages: torch.Tensor, table: torch.Tensor, page_size: int, head_dim: int):
        if pages.dim() != 3 or pages.dtype != torch.uint8 or pages.shape[2] != page_size * (head_dim + 8):
            raise MoEError("pages: expected uint8 [n_pages, n_kv_heads, page_size * (head_dim + 8)]")
        if table.dim() != 2 or table.dtype != torch.int32:
            raise MoEError("table: expected int32 [n_seq, max_pages]")
        if pages.device != table.device:
            raise MoEError("pages and table are on different devices")
        self.pages, self.table = pages, table
        self.page_size, self.head_dim = page_size, head_dim
        self.n_kv_heads, self.n_seq = pages.shape[1], table.shape[0]
        self.max_slots = table.shape[1] * page_size
        self.device = pages.device
        self._struct = L.Kv4CacheStruct(pages.shape[0], page_size, pages.shape[1], head_dim, table.shape[0],
                                        table.shape[1], _ptr(pages), _ptr(table))

    @classmethod
    def new(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, n_seq: int, max_pages: int,
            device="cuda") -> "Kv4Cache":
        """An empty cache; every table entry -1 (no page)."""
        pages = torch.empty((n_pages, n_kv_heads, page_size * (head_dim + 8)), dtype=torch.uint8, device=device)
        return cls(pages, torch.full((n_seq, max_pages), -1, dtype=torch.int32, device=device), page_size, head_dim)

    def new_mass(self) -> torch.Tensor:
        """Accumulated attention weights of every slot, zero: [n_seq, n_kv_heads, max_slots] fp32."""
        return torch.zeros((self.n_seq, self.n_kv_heads, self.max_slots), dtype=torch.float32, device=self.device)


def _strided(t: torch.Tensor, name: str, shape, dtype: Optional[torch.dtype] = None) -> int:
    """Pointer of a tensor whose last dimension is contiguous."""
    if not t.is_cuda:
        raise MoEError("expected a CUDA tensor")
    if t.dim() != 3 or tuple(t.shape) != tuple(shape):
        raise MoEError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise MoEError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise MoEError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr()


def _places(cache: Kv4Cache, seq: torch.Tensor, slot: torch.Tensor) -> int:
    if seq.dim() != 1:
        raise MoEError("seq: expected one dimension")
    T = seq.shape[0]
    _need(seq, torch.int32, (T,), "seq")
    _need(slot, torch.int32, (T,), "slot")
    return T


def kv4_append(cache: Kv4Cache, k: torch.Tensor, v: torch.Tensor, seq: torch.Tensor, slot: torch.Tensor,
               held: bool = False, dev_err: Optional[torch.Tensor] = None,
               stream=None) -> Optional[Tuple[torch.Tensor, torch.Tensor]]:
    """Quantises the keys and values of T tokens into their (seq, slot) places (slot -1: skipped).

    ``k`` and ``v`` [T, n_kv_heads, head_dim], bfloat16 or float32; token and head strides are free (multiples of
    16 bytes).  With ``held`` returns the values the cache now holds for them, same shape and type."""
    T = _places(cache, seq, slot)
    shape = (T, cache.n_kv_heads, cache.head_dim)
    dt = _DTYPES.get(k.dtype)
    if dt is None:
        raise MoEError(f"k: expected bfloat16 or float32, got {k.dtype}")
    kp, vp = _strided(k, "k", shape), _strided(v, "v", shape, k.dtype)
    out = (torch.empty(shape, dtype=k.dtype, device=k.device), torch.empty(shape, dtype=k.dtype, device=k.device)) if held else None
    ks, vs = k.stride(), v.stride()
    cfg = L.Kv4RowsCfg(T, dt, ks[0], ks[1], vs[0], vs[1])
    _check(L.load().kv4_append(C.byref(cache._struct), kp, vp, C.byref(cfg), _ptr(seq), _ptr(slot),
                               out[0].data_ptr() if held else None, out[1].data_ptr() if held else None,
                               _ptr(dev_err), _stream(stream)), "kv4_append")
    return out


def kv4_read(cache: Kv4Cache, seq: torch.Tensor, slot: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
             dev_err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The held keys and values [T, n_kv_heads, head_dim] of T (seq, slot) places (slot -1: zeros)."""
    T = _places(cache, seq, slot)
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise MoEError(f"dtype: expected bfloat16 or float32, got {dtype}")
    shape = (T, cache.n_kv_heads, cache.head_dim)
    k, v = torch.empty(shape, dtype=dtype, device=cache.device), torch.empty(shape, dtype=dtype, device=cache.device)
    cfg = L.Kv4RowsCfg(T, dt, 0, 0, 0, 0)
    _check(L.load().kv4_read(C.byref(cache._struct), _ptr(seq), _ptr(slot), C.byref(cfg), k.data_ptr(), v.data_ptr(),
                             _ptr(dev_err), _stream(stream)), "kv4_read")
    return k, v


def _attn(cache: Kv4Cache, q, q_start, base, max_q, visible, scale):
    if q.dim() != 3:
        raise MoEError("q: expected [T, n_q_heads, head_dim]")
    T, Hq, _ = q.shape
    qp = _strided(q, "q", (T, Hq, cache.head_dim), torch.bfloat16)
    _need(q_start, torch.int32, (cache.n_seq + 1,), "q_start")
    _need(base, torch.int32, (cache.n_seq,), "base")
    if visible is not None:
        _need(visible, torch.int64, (T,), "visible")
    st = q.stride()
    return qp, L.Kv4AttnCfg(T, Hq, max_q, cache.head_dim ** -0.5 if scale is None else scale, st[0], st[1])


def kv4_attend(cache: Kv4Cache, q: torch.Tensor, q_start: torch.Tensor, base: torch.Tensor, max_q: int,
               visible: Optional[torch.Tensor] = None, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of the new tokens over the cache: (out [T, n_q_heads, head_dim] bf16, lse [T, n_q_heads] fp32).

    Sequence s's new tokens are rows ``q_start[s]`` .. ``q_start[s + 1] - 1`` of ``q`` (bf16, token and head strides
    multiples of 8), appended at slots ``base[s]`` and on; each sees the ``base[s]`` context slots and, of the new
    ones, those set in its 64-bit mask ``visible`` (int64 [T]; None: itself and those before it).  ``max_q``: the
    most new tokens of a sequence; it chooses the kernel.  ``scale``: head_dim ** -0.5 if None."""
    lib = L.load()
    qp, cfg = _attn(cache, q, q_start, base, max_q, visible, scale)
    T, Hq, D = q.shape
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    _need(out, torch.bfloat16, (T, Hq, D), "out")
    _need(lse, torch.float32, (T, Hq), "lse")
    if workspace is None:
        workspace = torch.empty(kv4_attend_workspace_bytes(cache, cfg), dtype=torch.uint8, device=q.device)
    _check(lib.kv4_attend(C.byref(cache._struct), qp, _ptr(q_start), _ptr(base), _ptr(visible), C.byref(cfg), _ptr(out),
                          _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(dev_err), _stream(stream)), "kv4_attend")
    return out, lse


def kv4_attend_workspace_bytes(cache: Kv4Cache, cfg: L.Kv4AttnCfg) -> int:
    return int(L.load().kv4_attend_workspace(C.byref(cache._struct), C.byref(cfg)))


def kv4_weigh(cache: Kv4Cache, q: torch.Tensor, q_start: torch.Tensor, base: torch.Tensor, max_q: int,
              lse: torch.Tensor, mass: torch.Tensor, visible: Optional[torch.Tensor] = None,
              scale: Optional[float] = None, dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Adds to ``mass`` [n_seq, n_kv_heads, max_slots] the softmax weight that the new tokens gave each slot
    (arguments as kv4_attend, ``lse`` its result); returns ``mass``."""
    qp, cfg = _attn(cache, q, q_start, base, max_q, visible, scale)
    _need(lse, torch.float32, q.shape[:2], "lse")
    _need(mass, torch.float32, (cache.n_seq, cache.n_kv_heads, cache.max_slots), "mass")
    _check(L.load().kv4_weigh(C.byref(cache._struct), qp, _ptr(q_start), _ptr(base), _ptr(visible), _ptr(lse),
                              C.byref(cfg), _ptr(mass), _ptr(dev_err), _stream(stream)), "kv4_weigh")
    return mass


def kv4_evict(cache: Kv4Cache, mass: torch.Tensor, lens: torch.Tensor, keep: int, recent: int,
              mass_out: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
              stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Keeps, per sequence and kv head, the last ``recent`` slots and the others of largest mass, ``keep`` in all, and
    moves them to slots 0.. in their old order.  Returns (new_len [n_seq], origin [n_seq, n_kv_heads, keep]: the old
    slot of each new one, -1 past new_len, the masses: ``mass_out``, or ``mass`` itself rewritten where None)."""
    shape = (cache.n_seq, cache.n_kv_heads, cache.max_slots)
    _need(mass, torch.float32, shape, "mass")
    _need(lens, torch.int32, (cache.n_seq,), "lens")
    if mass_out is None:
        mass_out = mass
    _need(mass_out, torch.float32, shape, "mass_out")
    if keep < 1 or not 0 <= recent <= keep:
        raise MoEError("expected 1 <= keep and 0 <= recent <= keep")
    new_len = torch.empty(cache.n_seq, dtype=torch.int32, device=cache.device)
    origin = torch.empty((cache.n_seq, cache.n_kv_heads, keep), dtype=torch.int32, device=cache.device)
    cfg = L.Kv4EvictCfg(keep, recent)
    _check(L.load().kv4_evict(C.byref(cache._struct), _ptr(mass), _ptr(lens), C.byref(cfg), _ptr(new_len), _ptr(origin),
                              _ptr(mass_out), _ptr(dev_err), _stream(stream)), "kv4_evict")
    return new_len, origin, mass_out
