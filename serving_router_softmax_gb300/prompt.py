"""Binding of a prompt's pass through a layer (moe_rotate, moe_prompt_attend, moe_group_* of include/moe_verify.h).

Thin like ``api``: argument checks and pointer marshalling.  Tensors are on one CUDA device, whichever is current; calls
enqueue on that device's current stream (or ``stream``) and raise ``MoEError`` on a non-OK host status.  Device-side error
bits land in ``dev_err`` where one is given.  A small call's host time is of the order of its device time, so what follows
from the shapes of a call alone is kept.
"""
from __future__ import annotations

import ctypes as C
from typing import Dict, Optional, Sequence, Tuple

import torch

from . import _lib as L
from .api import LAYOUTS, ExpertLayer, MoEError, _check
from .kv4 import _DTYPES, _arg, _current_device, _err, _raw_stream

# 2 pi to 60 digits.
_TURN, _TURN_UNIT = 6283185307179586476925286766559005768394338798750211641949889, 10 ** 60


def _part_of_turn(f: float) -> int:
    """f / (2 pi), times 2^64, to the nearest whole number, mod 2^64, as a signed 64-bit number (f is taken as it is)."""
    a, b = f.as_integer_ratio()
    d = b * _TURN
    return ((((a << 65) * _TURN_UNIT + d) // (2 * d) + (1 << 63)) & ((1 << 64) - 1)) - (1 << 63)


# What is worked out from shapes, strides and types alone (no pointers).
_plans: Dict[tuple, tuple] = {}


def _plan(key: tuple, make) -> tuple:
    p = _plans.get(key)
    if p is None:
        if len(_plans) > 1024:
            _plans.clear()
        p = _plans[key] = make()
    return p


def _elsewhere(dev: int, stream, call):
    """`call` with device `dev` as the current one and `stream`, if there is one, as its stream (outputs are allocated there too)."""
    if dev < 0:
        raise MoEError("expected CUDA tensors")
    if stream is not None and stream.device_index != dev:
        raise MoEError(f"stream: expected one of cuda:{dev}")
    with torch.cuda.device(dev):
        if stream is None:
            return call()
        with torch.cuda.stream(stream):
            return call()


def _rows(t: torch.Tensor, name: str, shape, dtype: torch.dtype) -> Tuple[int, int]:
    """Token and head strides of a tensor [tokens, heads, dim] whose last dimension is contiguous."""
    if t.shape != shape:
        raise MoEError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise MoEError(f"{name}: dtype {t.dtype}, expected {dtype}")
    st = t.stride()
    if st[2] != 1 and shape[2] > 1:
        raise MoEError(f"{name}: the last dimension must be contiguous")
    return st[0], st[1]


def _ptr(dev: int, t: torch.Tensor, name: str) -> int:
    if t.get_device() != dev:
        raise MoEError(f"{name}: expected a tensor on cuda:{dev}")
    return t.data_ptr()


class Rotary:
    """Angles of a rotary position embedding: ``freqs[i]`` radians a position for pair i (the first 2 * len(freqs) of
    ``head_dim`` dimensions turn, the rest are copied) and ``axes[i]``, the axis whose positions it takes (None: axis 0).
    Pair i is dimensions (i, i + len(freqs)), or (2i, 2i + 1) with ``interleaved``."""

    def __init__(self, freqs: Sequence[float], head_dim: int, axes: Optional[Sequence[int]] = None, interleaved: bool = False,
                 device="cuda"):
        freqs = [float(f) for f in (freqs.tolist() if isinstance(freqs, torch.Tensor) else freqs)]
        axes = [0] * len(freqs) if axes is None else [int(x) for x in (axes.tolist() if isinstance(axes, torch.Tensor) else axes)]
        if len(axes) != len(freqs):
            raise MoEError("axes: expected one for each frequency")
        if not freqs or len(freqs) % 8 or 2 * len(freqs) > head_dim or head_dim % 8 or head_dim > 512:
            raise MoEError("freqs: expected a multiple of 8, at most head_dim / 2; head_dim a multiple of 8 up to 512")
        if min(axes) < 0 or max(axes) > 3:
            raise MoEError("axes: expected 0 to 3")
        if not all(abs(f) < float("inf") for f in freqs):
            raise MoEError("freqs: expected finite numbers")
        self.head_dim, self.rotary_dim, self.n_axes, self.interleaved = head_dim, 2 * len(freqs), max(axes) + 1, bool(interleaved)
        # (One copy: the turns, and behind them the axes, two to a word.)
        n = len(freqs)
        words = torch.tensor([_part_of_turn(f) for f in freqs] + [a | b << 32 for a, b in zip(axes[::2], axes[1::2])], dtype=torch.int64).to(device)
        self._turns, self._axis = words[:n], words[n:].view(torch.int32)
        self.device = self._turns.device

    @classmethod
    def standard(cls, head_dim: int, base: float = 10000.0, sections: Optional[Sequence[int]] = None,
                 rotary_dim: Optional[int] = None, interleaved: bool = False, device="cuda") -> "Rotary":
        """freqs[i] = base ** (-2 i / rotary_dim); ``sections``: how many pairs, in order, take each axis."""
        n, odd = divmod(head_dim if rotary_dim is None else rotary_dim, 2)
        if odd:
            raise MoEError("rotary_dim: expected an even number")
        if sections is not None and sum(sections) != n:
            raise MoEError(f"sections: expected a sum of {n}")
        axes = None if sections is None else [a for a, m in enumerate(sections) for _ in range(m)]
        return cls([base ** (-i / n) for i in range(n)], head_dim, axes, interleaved, device)


def rotate(rot: Rotary, q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, inverse: bool = False,
           out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None,
           dev_err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotates ``q`` [T, n_q_heads, head_dim] and ``k`` [T, n_k_heads, head_dim] (or None), bfloat16 or float32, by the
    positions ``pos`` (int32 [n_axes, T], or [T] with one axis); ``inverse`` turns back (the gradient).  Token and head
    strides are free (multiples of 16 bytes).  ``out_q`` / ``out_k``: may be q / k themselves; new tensors if None."""
    dev = q.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(dev, stream, lambda: rotate(rot, q, k, pos, inverse, out_q, out_k, dev_err))
    if rot.device.index != dev:
        raise MoEError(f"q: expected a tensor on {rot.device}")
    qs, ks = q.shape, None if k is None else k.shape
    inverse = bool(inverse)  # (a tensor would be looked up by its identity, whatever it holds)

    def make():
        if q.dim() != 3 or (k is not None and k.dim() != 3):
            raise MoEError("q, k: expected [T, heads, head_dim]")
        if q.dtype not in _DTYPES:
            raise MoEError(f"q: expected bfloat16 or float32, got {q.dtype}")
        T, Hq, D = qs[0], qs[1], rot.head_dim
        Hk = 0 if k is None else ks[1]
        strides = [*_rows(q, "q", (T, Hq, D), q.dtype), *((0, 0) if k is None else _rows(k, "k", (T, Hk, D), q.dtype))]
        strides += (Hq * D, D) if out_q is None else _rows(out_q, "out_q", qs, q.dtype)
        strides += (0, 0) if k is None else (Hk * D, D) if out_k is None else _rows(out_k, "out_k", ks, q.dtype)
        cfg = L.RotateCfg(T, Hq, Hk, D, rot.rotary_dim, rot.n_axes, int(rot.interleaved), int(inverse), _DTYPES[q.dtype], *strides)
        return C.byref(cfg), (T,), (rot.n_axes, T), strides[:4] == strides[4:]

    key = ("rotate", qs, q.stride(), q.dtype, ks, None if k is None else (k.stride(), k.dtype), rot.head_dim, rot.rotary_dim, rot.n_axes,
           rot.interleaved, inverse, None if out_q is None else (out_q.shape, out_q.stride(), out_q.dtype),
           None if out_k is None else (out_k.shape, out_k.stride(), out_k.dtype))
    ref, one, many, alike = _plan(key, make)
    oq = torch.empty(qs, dtype=q.dtype, device=q.device) if out_q is None else out_q
    ok = None if k is None else torch.empty(ks, dtype=k.dtype, device=k.device) if out_k is None else out_k
    qp, oqp = q.data_ptr(), _ptr(dev, oq, "out_q")
    kp, okp = (None, None) if k is None else (_ptr(dev, k, "k"), _ptr(dev, ok, "out_k"))
    if not alike and qs[0] and (qp == oqp and q.stride() != oq.stride() or k is not None and kp == okp and k.stride() != ok.stride()):
        raise MoEError("out_q, out_k: expected q and k themselves or memory apart from them")
    pp = _arg(dev, pos, torch.int32, one if rot.n_axes == 1 and pos.dim() == 1 else many, "pos")
    _check(L.load().moe_rotate(qp, kp, pp, rot._turns.data_ptr(), rot._axis.data_ptr(), ref, oqp, okp, _err(dev, dev_err),
                               _raw_stream(dev)), "moe_rotate")
    return oq, ok


def prompt_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, start: torch.Tensor, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  dev_err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention of packed prompts: (out [T, n_q_heads, head_dim] bf16, lse [T, n_q_heads] fp32).

    Sequence s is rows ``start[s]`` .. ``start[s + 1] - 1`` (int32 [n_seq + 1]) of ``q`` [T, n_q_heads, head_dim] and of
    ``k`` and ``v`` [T, n_kv_heads, head_dim] (bf16, token and head strides multiples of 8).  Rows of no sequence are left
    as they are.  ``scale``: head_dim ** -0.5 if None."""
    dev = q.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(dev, stream, lambda: prompt_attend(q, k, v, start, scale, out, lse, dev_err))
    if scale is not None:
        scale = float(scale)  # (as inverse, above)

    def make():
        if q.dim() != 3 or k.dim() != 3:
            raise MoEError("q, k, v: expected [T, heads, head_dim]")
        if start.dim() != 1 or start.shape[0] < 1:
            raise MoEError("start: expected int32 [n_seq + 1]")
        T, Hq, D = q.shape
        shape = (T, k.shape[1], D)
        cfg = L.PromptCfg(T, start.shape[0] - 1, Hq, k.shape[1], D, D ** -0.5 if scale is None else scale,
                          *_rows(q, "q", q.shape, torch.bfloat16), *_rows(k, "k", shape, torch.bfloat16),
                          *_rows(v, "v", shape, torch.bfloat16))
        return C.byref(cfg), (T, Hq, D), (T, Hq), start.shape

    ref, so, sl, ss = _plan(("attend", q.shape, q.stride(), q.dtype, k.shape, k.stride(), k.dtype, v.shape, v.stride(), v.dtype,
                             start.shape, scale), make)
    qp, kp, vp = q.data_ptr(), _ptr(dev, k, "k"), _ptr(dev, v, "v")
    o = torch.empty(so, dtype=torch.bfloat16, device=q.device) if out is None else out
    z = torch.empty(sl, dtype=torch.float32, device=q.device) if lse is None else lse
    _check(L.load().moe_prompt_attend(qp, kp, vp, _arg(dev, start, torch.int32, ss, "start"), ref,
                                      o.data_ptr() if out is None else _arg(dev, o, torch.bfloat16, so, "out"),
                                      z.data_ptr() if lse is None else _arg(dev, z, torch.float32, sl, "lse"),
                                      _err(dev, dev_err), _raw_stream(dev)), "moe_prompt_attend")
    return o, z


def _group_plan(rows: int, k: int, layer: ExpertLayer) -> tuple:
    """What a layer's struct begins with; shapes of x, h, y, w, and of the union's n_unique, unique, offsets and lists."""
    gu, dn, pool = layer.gate_up, layer.down, layer.pool

    def make():
        if layer.dtype != "bf16":
            raise MoEError(f"layer: expected bf16 weights, got {layer.dtype}")
        if k < 1 or rows % k:
            raise MoEError(f"expected k >= 1 rows of each token, got {rows} for k = {k}")
        H, I, E = layer.H, layer.I, layer.E
        # Bytes of an expert's matrices (tiled: the rows of gate, of up and of down, each rounded up to 128).
        up = 128 if layer.layout == "tiled" else 1
        slots = E if pool is None else pool.n_slots
        for t, name, n in ((gu, "gate_up", 4 * (-(-I // up) * up) * H), (dn, "down", 2 * (-(-H // up) * up) * I)):
            if t.numel() * t.dtype.itemsize < slots * n:
                raise MoEError(f"layer: {name} holds {t.numel() * t.dtype.itemsize} bytes of {slots * n}")
        T, cap = rows // k, min(E, rows)
        head = (H, I, E, L.DTYPE_BF16, LAYOUTS[layer.layout])
        return head, (T, H), (rows, I), (T, H), (T, k), (1,), (max(cap, 1),), (cap + 1,), (max(rows, 1),)

    return _plan(("group", rows, k, gu.shape, gu.dtype, dn.shape, dn.dtype, layer.dims, layer.dtype, layer.layout,
                  None if pool is None else pool.n_slots), make)


def _layer_on(dev: int, layer: ExpertLayer, head: tuple):
    """The layer's struct (without a pool in 2 us instead of 5)."""
    gu, dn = layer.gate_up, layer.down
    if gu.get_device() != dev or dn.get_device() != dev or not gu.is_contiguous() or not dn.is_contiguous():
        raise MoEError(f"layer: expected contiguous weights on cuda:{dev}")
    return C.byref(L.LayerWeights(*head, gu.data_ptr(), dn.data_ptr()) if layer.pool is None else layer.struct())


def group_gate_up(x: torch.Tensor, layer: ExpertLayer, union: Dict[str, torch.Tensor], k: int, out: Optional[torch.Tensor] = None,
                  dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """h [T * k, I] bf16: silu(W_gate x) * (W_up x) for every row of the groups of ``union`` (``union_permute``'s, for the
    same T tokens' k experts), in the groups' order.  ``x`` [T, H] bf16; ``layer``: bf16, either layout.  T * k may be up to
    2^22; ``union_permute`` takes T * k <= 65536 and T * ceil(E / 32) <= 32768, so more tokens go through in parts."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(dev, stream, lambda: group_gate_up(x, layer, union, k, out, dev_err))
    T = x.shape[0]
    head, sx, sh, _, _, s1, su, so, sp = _group_plan(T * k, k, layer)
    ref = _layer_on(dev, layer, head)
    h = torch.empty(sh, dtype=torch.bfloat16, device=x.device) if out is None else out
    i32 = torch.int32
    _check(L.load().moe_group_gate_up(_arg(dev, x, torch.bfloat16, sx, "x"), T, k, ref, _arg(dev, union["n_unique"], i32, s1, "n_unique"),
                                      _arg(dev, union["unique"], i32, su, "unique"), _arg(dev, union["offsets"], i32, so, "offsets"),
                                      _arg(dev, union["perm_token"], i32, sp, "perm_token"),
                                      h.data_ptr() if out is None else _arg(dev, h, torch.bfloat16, sh, "out"), _err(dev, dev_err),
                                      _raw_stream(dev)), "moe_group_gate_up")
    return h


def group_down_workspace_bytes(layer: ExpertLayer, T: int, k: int) -> int:
    """Bytes of workspace that group_down needs for T tokens of k experts each."""
    st = layer.struct()
    return int(L.load().moe_group_down_workspace(C.byref(st), T, k))


def group_down(h: torch.Tensor, layer: ExpertLayer, union: Dict[str, torch.Tensor], w: torch.Tensor, y: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [T, H] bf16 = sum_j w[t, j] * (W_down h[inv[t, j]]): ``h`` [T * k, I] bf16 in the groups' order (``group_gate_up``'s),
    ``w`` [T, k] fp32 routing weights.  The terms are rounded to bf16 before they are summed in fp32: ``y`` is off by up to
    2^-8 of the sum of their sizes (``verify_ffn`` keeps them in fp32)."""
    dev = h.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(dev, stream, lambda: group_down(h, layer, union, w, y, workspace, dev_err))
    if w.dim() != 2:
        raise MoEError("w: expected [T, k]")
    T, k = w.shape
    head, _, sh, sy, sw, s1, su, so, sp = _group_plan(T * k, k, layer)
    ref = _layer_on(dev, layer, head)
    o = torch.empty(sy, dtype=torch.bfloat16, device=h.device) if y is None else y
    lib, i32 = L.load(), torch.int32
    if workspace is None:
        workspace = torch.empty((lib.moe_group_down_workspace(ref, T, k),), dtype=torch.uint8, device=h.device)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise MoEError(f"workspace: expected contiguous bytes (uint8) on cuda:{dev}")
    _check(lib.moe_group_down(_arg(dev, h, torch.bfloat16, sh, "h"), T, k, ref, _arg(dev, union["n_unique"], i32, s1, "n_unique"),
                              _arg(dev, union["unique"], i32, su, "unique"), _arg(dev, union["offsets"], i32, so, "offsets"),
                              _arg(dev, union["inv"], i32, sp, "inv"), _arg(dev, w, torch.float32, sw, "w"),
                              o.data_ptr() if y is None else _arg(dev, o, torch.bfloat16, sy, "y"), workspace.data_ptr(),
                              workspace.numel(), _err(dev, dev_err), _raw_stream(dev)), "moe_group_down")
    return o
