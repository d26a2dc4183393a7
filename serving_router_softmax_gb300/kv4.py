"""Binding of the 4-bit paged KV cache (kv4_* of include/moe_verify.h).

Thin like ``api``: argument checks and pointer marshalling; tensors are on the
cache's CUDA device, whichever is current, calls enqueue on that device's
current stream (or ``stream``) and raise ``MoEError`` on a non-OK host status.
Device-side error bits land in ``dev_err`` where one is given.

A small call's host time is of the order of its device time, so what does not
change from call to call is kept: the argument structs with the cache, and one
workspace for each stream and host thread.  A thread's calls on a stream follow
each other, so the caches of all layers share it; another thread's may come
between the two launches of a kv4_attend.
"""
from __future__ import annotations

import ctypes as C
import threading
from typing import Optional, Tuple

import torch

from . import _lib as L
from .api import MoEError, _check, _need

_DTYPES = {torch.float32: L.DTYPE_F32, torch.bfloat16: L.DTYPE_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device

_STREAMS_KEPT = 16


class _Workspaces(threading.local):
    def __init__(self):
        self.held = {}  # (device, stream) -> the largest workspace that this thread's calls there have needed


_workspaces = _Workspaces()


def _workspace(index: int, nbytes: int, stream: int) -> torch.Tensor:
    # A graph's calls must not share a workspace with calls that may run beside its replays.
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
    held = _workspaces.held
    w = held.get((index, stream))
    if w is None or w.numel() < nbytes:
        # (What is dropped goes back to the allocator's blocks of its own stream, behind the calls that use it.)
        if w is None and len(held) >= _STREAMS_KEPT:
            del held[next(iter(held))]
        w = held[index, stream] = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
    return w


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
        for t in (pages, table):
            if not t.is_cuda or not t.is_contiguous():
                raise MoEError("expected contiguous CUDA tensors")
        self.pages, self.table = pages, table
        self.page_size, self.head_dim = page_size, head_dim
        self.n_kv_heads, self.n_seq = pages.shape[1], table.shape[0]
        self.max_slots = table.shape[1] * page_size
        self.device, self._index = pages.device, pages.device.index
        self._struct = L.Kv4CacheStruct(pages.shape[0], page_size, pages.shape[1], head_dim, table.shape[0],
                                        table.shape[1], pages.data_ptr(), table.data_ptr())
        self._ref = C.byref(self._struct)
        self._plans = {}

    @classmethod
    def new(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, n_seq: int, max_pages: int,
            device="cuda") -> "Kv4Cache":
        """An empty cache; every table entry -1 (no page)."""
        pages = torch.empty((n_pages, n_kv_heads, page_size * (head_dim + 8)), dtype=torch.uint8, device=device)
        return cls(pages, torch.full((n_seq, max_pages), -1, dtype=torch.int32, device=device), page_size, head_dim)

    def new_mass(self) -> torch.Tensor:
        """Accumulated attention weights of every slot, zero: [n_seq, n_kv_heads, max_slots] fp32."""
        return torch.zeros((self.n_seq, self.n_kv_heads, self.max_slots), dtype=torch.float32, device=self.device)

    def _plan(self, key, make):
        """The argument struct (and what else `make` gives) of calls of one shape."""
        p = self._plans.get(key)
        if p is None:
            if len(self._plans) > 256:
                self._plans.clear()
            p = self._plans[key] = make()
        return p


def _arg(index: int, t: torch.Tensor, dtype: torch.dtype, shape, name: str) -> int:
    """Pointer of a contiguous tensor of device `index`, of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _need(t, dtype, shape, name)
        raise MoEError(f"{name}: expected a contiguous tensor on cuda:{index}")
    return t.data_ptr()


def _err(index: int, t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else _arg(index, t, torch.int32, (1,), "dev_err")


def _strided(index: int, t: torch.Tensor, name: str, shape, dtype: torch.dtype) -> None:
    """A tensor of device `index` whose last dimension is contiguous."""
    if t.get_device() != index:
        raise MoEError(f"{name}: expected a tensor on cuda:{index}")
    if t.dim() != 3 or t.shape != shape:
        raise MoEError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise MoEError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise MoEError(f"{name}: the last dimension must be contiguous")


def _on(stream, call, cache: Kv4Cache, *args):
    """The call with the cache's device as the current one and `stream`, if there is one, as its stream: its outputs and
    workspace are allocated there too."""
    if stream is not None and stream.device_index != cache._index:
        raise MoEError(f"stream: expected one of cuda:{cache._index}")
    with torch.cuda.device(cache._index):
        if stream is None:
            return call(cache, *args)
        with torch.cuda.stream(stream):
            return call(cache, *args)


def kv4_append(cache: Kv4Cache, k: torch.Tensor, v: torch.Tensor, seq: torch.Tensor, slot: torch.Tensor,
               held: bool = False, dev_err: Optional[torch.Tensor] = None,
               stream=None) -> Optional[Tuple[torch.Tensor, torch.Tensor]]:
    """Quantises the keys and values of T tokens into their (seq, slot) places (slot -1: skipped).

    ``k`` and ``v`` [T, n_kv_heads, head_dim], bfloat16 or float32; token and head strides are free (multiples of
    16 bytes).  With ``held`` returns the values the cache now holds for them, same shape and type."""
    if stream is not None or _current_device() != cache._index:
        return _on(stream, kv4_append, cache, k, v, seq, slot, held, dev_err)
    dev = cache._index
    T = seq.shape[0] if seq.dim() == 1 else -1

    def make():
        shape = (T, cache.n_kv_heads, cache.head_dim)
        if k.dtype not in _DTYPES:
            raise MoEError(f"k: expected bfloat16 or float32, got {k.dtype}")
        _strided(cache._index, k, "k", shape, k.dtype)
        _strided(cache._index, v, "v", shape, k.dtype)
        ks, vs = k.stride(), v.stride()
        cfg = L.Kv4RowsCfg(T, _DTYPES[k.dtype], ks[0], ks[1], vs[0], vs[1])
        return C.byref(cfg), shape

    ref, shape = cache._plan(("append", T, k.dtype, v.dtype, k.shape, v.shape, k.stride(), v.stride(), k.get_device(),
                              v.get_device()), make)
    kh = vh = None
    if held:
        kh = torch.empty(shape, dtype=k.dtype, device=cache.device)
        vh = torch.empty(shape, dtype=k.dtype, device=cache.device)
    _check(L.load().kv4_append(cache._ref, k.data_ptr(), v.data_ptr(), ref, _arg(dev, seq, torch.int32, (T,), "seq"),
                               _arg(dev, slot, torch.int32, (T,), "slot"), kh.data_ptr() if held else None,
                               vh.data_ptr() if held else None, _err(dev, dev_err), _raw_stream(cache._index)), "kv4_append")
    return (kh, vh) if held else None


def kv4_read(cache: Kv4Cache, seq: torch.Tensor, slot: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
             dev_err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The held keys and values [T, n_kv_heads, head_dim] of T (seq, slot) places (slot -1: zeros)."""
    if stream is not None or _current_device() != cache._index:
        return _on(stream, kv4_read, cache, seq, slot, dtype, dev_err)
    dev = cache._index
    T = seq.shape[0] if seq.dim() == 1 else -1

    def make():
        if dtype not in _DTYPES:
            raise MoEError(f"dtype: expected bfloat16 or float32, got {dtype}")
        return C.byref(L.Kv4RowsCfg(T, _DTYPES[dtype], 0, 0, 0, 0)), (T, cache.n_kv_heads, cache.head_dim)

    sp, jp = _arg(dev, seq, torch.int32, (T,), "seq"), _arg(dev, slot, torch.int32, (T,), "slot")
    ref, shape = cache._plan(("read", T, dtype), make)
    k = torch.empty(shape, dtype=dtype, device=cache.device)
    v = torch.empty(shape, dtype=dtype, device=cache.device)
    _check(L.load().kv4_read(cache._ref, sp, jp, ref, k.data_ptr(), v.data_ptr(), _err(dev, dev_err),
                             _raw_stream(cache._index)), "kv4_read")
    return k, v


def _attn_plan(cache: Kv4Cache, q: torch.Tensor, max_q: int, scale: Optional[float]):
    """(struct, workspace bytes, shapes of out, lse, q_start, base, visible) of a call with these queries."""
    if scale is not None:
        scale = float(scale)  # (a tensor would be looked up by its identity, whatever it holds)

    def make():
        if q.dim() != 3:
            raise MoEError("q: expected [T, n_q_heads, head_dim]")
        T, Hq, _ = q.shape
        _strided(cache._index, q, "q", (T, Hq, cache.head_dim), torch.bfloat16)
        st = q.stride()
        cfg = L.Kv4AttnCfg(T, Hq, max_q, cache.head_dim ** -0.5 if scale is None else scale, st[0], st[1])
        ref = C.byref(cfg)
        return (ref, int(L.load().kv4_attend_workspace(cache._ref, ref)), (T, Hq, cache.head_dim), (T, Hq),
                (cache.n_seq + 1,), (cache.n_seq,), (T,))

    return cache._plan(("attn", q.shape, q.stride(), q.dtype, q.get_device(), max_q, scale), make)


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
    if stream is not None or _current_device() != cache._index:
        return _on(stream, kv4_attend, cache, q, q_start, base, max_q, visible, scale, out, lse, workspace, dev_err)
    dev = cache._index
    ref, need, so, sl, sq, sb, sv = _attn_plan(cache, q, max_q, scale)
    if out is None:
        out = torch.empty(so, dtype=torch.bfloat16, device=cache.device)
    if lse is None:
        lse = torch.empty(sl, dtype=torch.float32, device=cache.device)
    st = _raw_stream(cache._index)
    if workspace is None:
        workspace = _workspace(cache._index, need, st)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != cache._index or not workspace.is_contiguous():
        raise MoEError(f"workspace: expected contiguous bytes (uint8) on cuda:{cache._index}")
    _check(L.load().kv4_attend(cache._ref, q.data_ptr(), _arg(dev, q_start, torch.int32, sq, "q_start"),
                               _arg(dev, base, torch.int32, sb, "base"),
                               None if visible is None else _arg(dev, visible, torch.int64, sv, "visible"), ref,
                               _arg(dev, out, torch.bfloat16, so, "out"), _arg(dev, lse, torch.float32, sl, "lse"),
                               workspace.data_ptr(), workspace.numel(), _err(dev, dev_err), st), "kv4_attend")
    return out, lse


def kv4_attend_workspace_bytes(cache: Kv4Cache, q: torch.Tensor, max_q: int) -> int:
    """Bytes of workspace that kv4_attend needs for queries of this shape."""
    if _current_device() != cache._index:
        return _on(None, kv4_attend_workspace_bytes, cache, q, max_q)
    return _attn_plan(cache, q, max_q, None)[1]


def kv4_weigh(cache: Kv4Cache, q: torch.Tensor, q_start: torch.Tensor, base: torch.Tensor, max_q: int,
              lse: torch.Tensor, mass: torch.Tensor, visible: Optional[torch.Tensor] = None,
              scale: Optional[float] = None, dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Adds to ``mass`` [n_seq, n_kv_heads, max_slots] the softmax weight that the new tokens gave each slot
    (arguments as kv4_attend, ``lse`` its result); returns ``mass``."""
    if stream is not None or _current_device() != cache._index:
        return _on(stream, kv4_weigh, cache, q, q_start, base, max_q, lse, mass, visible, scale, dev_err)
    dev = cache._index
    ref, _, _, sl, sq, sb, sv = _attn_plan(cache, q, max_q, scale)
    _check(L.load().kv4_weigh(cache._ref, q.data_ptr(), _arg(dev, q_start, torch.int32, sq, "q_start"),
                              _arg(dev, base, torch.int32, sb, "base"),
                              None if visible is None else _arg(dev, visible, torch.int64, sv, "visible"),
                              _arg(dev, lse, torch.float32, sl, "lse"), ref,
                              _arg(dev, mass, torch.float32, (cache.n_seq, cache.n_kv_heads, cache.max_slots), "mass"),
                              _err(dev, dev_err), _raw_stream(cache._index)), "kv4_weigh")
    return mass


def kv4_evict(cache: Kv4Cache, mass: torch.Tensor, lens: torch.Tensor, keep: int, recent: int,
              mass_out: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
              stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Keeps, per sequence and kv head, the last ``recent`` slots and the others of largest mass, ``keep`` in all, and
    moves them to slots 0.. in their old order.  Returns (new_len [n_seq], origin [n_seq, n_kv_heads, keep]: the old
    slot of each new one, -1 past new_len, the masses: ``mass_out``, or ``mass`` itself rewritten where None)."""
    if stream is not None or _current_device() != cache._index:
        return _on(stream, kv4_evict, cache, mass, lens, keep, recent, mass_out, dev_err)
    dev = cache._index

    def make():
        if keep < 1 or not 0 <= recent <= keep:
            raise MoEError("expected 1 <= keep and 0 <= recent <= keep")
        return (C.byref(L.Kv4EvictCfg(keep, recent)), (cache.n_seq, cache.n_kv_heads, cache.max_slots), (cache.n_seq,),
                (cache.n_seq, cache.n_kv_heads, keep))

    ref, sm, sn, so = cache._plan(("evict", keep, recent), make)
    if mass_out is None:
        mass_out = mass
    new_len = torch.empty(sn, dtype=torch.int32, device=cache.device)
    origin = torch.empty(so, dtype=torch.int32, device=cache.device)
    _check(L.load().kv4_evict(cache._ref, _arg(dev, mass, torch.float32, sm, "mass"), _arg(dev, lens, torch.int32, sn, "lens"), ref,
                              new_len.data_ptr(), origin.data_ptr(), _arg(dev, mass_out, torch.float32, sm, "mass_out"),
                              _err(dev, dev_err), _raw_stream(cache._index)), "kv4_evict")
    return new_len, origin, mass_out
