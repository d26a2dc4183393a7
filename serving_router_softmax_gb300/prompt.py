"""Binding of a prompt's pass through a layer (moe_rotate, moe_prompt_attend, moe_group_* of include/moe_verify.h).

Thin like ``api``: argument checks and pointer marshalling.  Tensors are on one CUDA device, whichever is current; calls
enqueue on that device's current stream (or ``stream``) and raise ``MoEError`` on a non-OK host status.  Device-side error
bits land in ``dev_err`` where one is given.
"""
from __future__ import annotations

import ctypes as C
from fractions import Fraction
from typing import Dict, Optional, Sequence, Tuple

import torch

from . import _lib as L
from .api import ExpertLayer, MoEError, _check
from .kv4 import _DTYPES, _arg, _current_device, _err, _raw_stream

# 2 pi to 60 digits.
_TURN = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def _run(dev: torch.device, stream, call):
    """The call with `dev` as the current device and `stream`, if there is one, as its stream (outputs are allocated there too)."""
    if dev.type != "cuda":
        raise MoEError("expected CUDA tensors")
    if stream is not None and stream.device_index != dev.index:
        raise MoEError(f"stream: expected one of {dev}")
    if stream is None and _current_device() == dev.index:
        return call(dev.index)
    with torch.cuda.device(dev.index):
        if stream is None:
            return call(dev.index)
        with torch.cuda.stream(stream):
            return call(dev.index)


def _rows(index: int, t: torch.Tensor, name: str, shape, dtype: torch.dtype) -> Tuple[int, int, int]:
    """(pointer, token stride, head stride) of a tensor [tokens, heads, dim] whose last dimension is contiguous."""
    if t.get_device() != index:
        raise MoEError(f"{name}: expected a tensor on cuda:{index}")
    if t.shape != shape:
        raise MoEError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise MoEError(f"{name}: dtype {t.dtype}, expected {dtype}")
    st = t.stride()
    if st[2] != 1 and shape[2] > 1:
        raise MoEError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), st[0], st[1]


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
        turns = [round(Fraction(f) / _TURN * 2 ** 64) % 2 ** 64 for f in freqs]
        self.head_dim, self.rotary_dim, self.n_axes, self.interleaved = head_dim, 2 * len(freqs), max(axes) + 1, bool(interleaved)
        self._turns = torch.tensor([t - 2 ** 64 if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self._axis = torch.tensor(axes, dtype=torch.int32, device=device)
        self.device = self._turns.device

    @classmethod
    def standard(cls, head_dim: int, base: float = 10000.0, sections: Optional[Sequence[int]] = None,
                 rotary_dim: Optional[int] = None, interleaved: bool = False, device="cuda") -> "Rotary":
        """freqs[i] = base ** (-2 i / rotary_dim); ``sections``: how many pairs, in order, take each axis."""
        n = (head_dim if rotary_dim is None else rotary_dim) // 2
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
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise MoEError("q, k: expected [T, heads, head_dim]")
    if q.dtype not in _DTYPES:
        raise MoEError(f"q: expected bfloat16 or float32, got {q.dtype}")
    if rot.device != q.device:
        raise MoEError(f"q: expected a tensor on {rot.device}")

    def call(dev: int):
        T, Hq = q.shape[:2]
        Hk = 0 if k is None else k.shape[1]
        qp, *qs = _rows(dev, q, "q", (T, Hq, rot.head_dim), q.dtype)
        kp, *ks = (None, 0, 0) if k is None else _rows(dev, k, "k", (T, Hk, rot.head_dim), q.dtype)
        oq = torch.empty(q.shape, dtype=q.dtype, device=q.device) if out_q is None else out_q
        ok = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device) if out_k is None else out_k
        oqp, *oqs = _rows(dev, oq, "out_q", q.shape, q.dtype)
        okp, *oks = (None, 0, 0) if k is None else _rows(dev, ok, "out_k", k.shape, q.dtype)
        for name, x, y, xp, yp, xs, ys in (("q", q, oq, qp, oqp, qs, oqs), ("k", k, ok, kp, okp, ks, oks)):
            if x is not None and xp == yp and xs != ys:
                raise MoEError(f"out_{name}: expected {name} itself or memory apart from it")
        pp = _arg(dev, pos, torch.int32, (T,) if pos.dim() == 1 and rot.n_axes == 1 else (rot.n_axes, T), "pos")
        cfg = L.RotateCfg(T, Hq, Hk, rot.head_dim, rot.rotary_dim, rot.n_axes, int(rot.interleaved), int(inverse), _DTYPES[q.dtype],
                          *qs, *ks, *oqs, *oks)
        _check(L.load().moe_rotate(qp, kp, pp, rot._turns.data_ptr(), rot._axis.data_ptr(), C.byref(cfg), oqp, okp,
                                   _err(dev, dev_err), _raw_stream(dev)), "moe_rotate")
        return oq, ok

    return _run(q.device, stream, call)


def prompt_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, start: torch.Tensor, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  dev_err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention of packed prompts: (out [T, n_q_heads, head_dim] bf16, lse [T, n_q_heads] fp32).

    Sequence s is rows ``start[s]`` .. ``start[s + 1] - 1`` (int32 [n_seq + 1]) of ``q`` [T, n_q_heads, head_dim] and of
    ``k`` and ``v`` [T, n_kv_heads, head_dim] (bf16, token and head strides multiples of 8).  Rows of no sequence are left
    as they are.  ``scale``: head_dim ** -0.5 if None."""
    if q.dim() != 3 or k.dim() != 3:
        raise MoEError("q, k, v: expected [T, heads, head_dim]")
    if start.dim() != 1 or start.shape[0] < 1:
        raise MoEError("start: expected int32 [n_seq + 1]")

    def call(dev: int):
        T, Hq, D = q.shape
        shape = (T, k.shape[1], D)
        qp, *qs = _rows(dev, q, "q", q.shape, torch.bfloat16)
        kp, *ks = _rows(dev, k, "k", shape, torch.bfloat16)
        vp, *vs = _rows(dev, v, "v", shape, torch.bfloat16)
        o = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device) if out is None else out
        z = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
        cfg = L.PromptCfg(T, start.shape[0] - 1, Hq, k.shape[1], D, D ** -0.5 if scale is None else scale, *qs, *ks, *vs)
        _check(L.load().moe_prompt_attend(qp, kp, vp, _arg(dev, start, torch.int32, start.shape, "start"), C.byref(cfg),
                                          _arg(dev, o, torch.bfloat16, (T, Hq, D), "out"), _arg(dev, z, torch.float32, (T, Hq), "lse"),
                                          _err(dev, dev_err), _raw_stream(dev)), "moe_prompt_attend")
        return o, z

    return _run(q.device, stream, call)


def _union_args(dev: int, union: Dict[str, torch.Tensor], names, rows: int, E: int):
    cap = min(E, rows)
    shapes = {"n_unique": (1,), "unique": (max(cap, 1),), "offsets": (cap + 1,), "perm_token": (max(rows, 1),), "inv": (max(rows, 1),)}
    return [_arg(dev, union[n], torch.int32, shapes[n], f"union[{n!r}]") for n in names]


def _layer(dev: int, layer: ExpertLayer) -> L.LayerWeights:
    if layer.gate_up.get_device() != dev or layer.down.get_device() != dev:
        raise MoEError(f"layer: expected one on cuda:{dev}")
    return layer.struct()


def group_gate_up(x: torch.Tensor, layer: ExpertLayer, union: Dict[str, torch.Tensor], k: int, out: Optional[torch.Tensor] = None,
                  dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """h [T * k, I] bf16: silu(W_gate x) * (W_up x) for every row of the groups of ``union`` (``union_permute``'s, for the
    same T tokens' k experts), in the groups' order.  ``x`` [T, H] bf16, any T; ``layer``: bf16, either layout."""
    if x.dim() != 2 or x.shape[1] != layer.H:
        raise MoEError("x: expected [T, H] of the layer's H")

    def call(dev: int):
        T = x.shape[0]
        if k < 1:
            raise MoEError("k < 1")
        st = _layer(dev, layer)
        h = torch.empty((T * k, layer.I), dtype=torch.bfloat16, device=x.device) if out is None else out
        args = _union_args(dev, union, ("n_unique", "unique", "offsets", "perm_token"), T * k, layer.E)
        _check(L.load().moe_group_gate_up(_arg(dev, x, torch.bfloat16, x.shape, "x"), T, k, C.byref(st), *args,
                                          _arg(dev, h, torch.bfloat16, (T * k, layer.I), "out"), _err(dev, dev_err), _raw_stream(dev)),
               "moe_group_gate_up")
        return h

    return _run(x.device, stream, call)


def group_down_workspace_bytes(layer: ExpertLayer, T: int, k: int) -> int:
    """Bytes of workspace that group_down needs for T tokens of k experts each."""
    st = layer.struct()
    return int(L.load().moe_group_down_workspace(C.byref(st), T, k))


def group_down(h: torch.Tensor, layer: ExpertLayer, union: Dict[str, torch.Tensor], w: torch.Tensor, y: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [T, H] bf16 = sum_j w[t, j] * (W_down h[inv[t, j]]): ``h`` [T * k, I] bf16 in the groups' order (``group_gate_up``'s),
    ``w`` [T, k] fp32 routing weights."""
    if h.dim() != 2 or w.dim() != 2:
        raise MoEError("h: expected [T * k, I], w: [T, k]")

    def call(dev: int):
        T, k = w.shape
        if k < 1:
            raise MoEError("w: expected [T, k]")
        st = _layer(dev, layer)
        o = torch.empty((T, layer.H), dtype=torch.bfloat16, device=h.device) if y is None else y
        ws = workspace
        if ws is None:
            ws = torch.empty(int(L.load().moe_group_down_workspace(C.byref(st), T, k)), dtype=torch.uint8, device=h.device)
        elif ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
            raise MoEError(f"workspace: expected contiguous bytes (uint8) on cuda:{dev}")
        args = _union_args(dev, union, ("n_unique", "unique", "offsets", "inv"), T * k, layer.E)
        _check(L.load().moe_group_down(_arg(dev, h, torch.bfloat16, (T * k, layer.I), "h"), T, k, C.byref(st), *args,
                                       _arg(dev, w, torch.float32, (T, k), "w"), _arg(dev, o, torch.bfloat16, (T, layer.H), "y"),
                                       ws.data_ptr(), ws.numel(), _err(dev, dev_err), _raw_stream(dev)), "moe_group_down")
        return o

    return _run(h.device, stream, call)
