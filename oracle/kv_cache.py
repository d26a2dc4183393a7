"""CPU oracle of the 4-bit paged KV cache (kv4_*), in 64 bits.

The S2-MoE write-up's component 2 keeps the draft's and the target's keys and
values in one cache; the entry format, the visibility masks and the eviction
rule checked here are the library's own (include/moe_verify.h).  Arrays are
numpy; pages are the raw bytes.
"""
from __future__ import annotations

import numpy as np


def quantise(x: np.ndarray):
    """Codes [..., D], scale and zero [...] (fp16 values as float64) of rows x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    lo, hi = x.min(-1), x.max(-1)
    ok = np.isfinite(x).all(-1) & (lo >= -65504) & (hi <= 65504)
    lo, hi = np.where(ok, lo, 0.0), np.where(ok, hi, 0.0)
    scale = ((hi - lo) / 15.0).astype(np.float32).astype(np.float16).astype(np.float64)
    zero = lo.astype(np.float32).astype(np.float16).astype(np.float64)
    safe = np.where(scale > 0, scale, 1.0)
    with np.errstate(invalid="ignore"):
        code = np.clip(np.rint((x - zero[..., None]) / safe[..., None]), 0, 15)
    code = np.where((scale > 0)[..., None] & ok[..., None], code, 0.0)
    return code.astype(np.uint8), np.where(ok, scale, 0.0), np.where(ok, zero, np.nan)


class Pages:
    """Views of raw pages uint8 [n_pages, Hkv, page * (D + 8)] (changes go through to it)."""

    def __init__(self, raw: np.ndarray, table: np.ndarray, page: int, D: int):
        self.raw, self.table, self.page, self.D = raw, table, page, D
        half = page * D // 2
        n, H = raw.shape[:2]
        self.codes = (raw[:, :, :half].reshape(n, H, page, D // 2), raw[:, :, half:2 * half].reshape(n, H, page, D // 2))
        self.par = raw[:, :, 2 * half:].view(np.float16).reshape(n, H, page, 4)

    def valid(self, s: int, n: int) -> np.ndarray:
        j = np.arange(n)
        p = self.table[s][j // self.page]
        return (p >= 0) & (p < self.raw.shape[0])

    def entries(self, s: int, h: int, n: int, part: int):
        """Codes [n, D], scale [n], zero [n] of the first n slots; rows of invalid pages are zeros."""
        j = np.arange(n)
        p = self.table[s][j // self.page]
        ok = (p >= 0) & (p < self.raw.shape[0])
        p = np.where(ok, p, 0)
        raw = self.codes[part][p, h, j % self.page]
        code = np.empty((n, self.D), dtype=np.float64)
        code[:, 0::2], code[:, 1::2] = raw & 15, raw >> 4
        par = self.par[p, h, j % self.page].astype(np.float64)
        return code * ok[:, None], np.where(ok, par[:, 2 * part], 0.0), np.where(ok, par[:, 2 * part + 1], 0.0)

    def write(self, s: int, slot: int, part: int, x: np.ndarray):
        """Rows x [Hkv, D] to a slot."""
        code, scale, zero = quantise(x)
        p, r = int(self.table[s][slot // self.page]), slot % self.page
        self.codes[part][p, :, r] = code[:, 0::2] | (code[:, 1::2] << 4)
        self.par[p, :, r, 2 * part], self.par[p, :, r, 2 * part + 1] = scale, zero


def seen(base: int, n: int, mask=None) -> np.ndarray:
    """[n, base + n]: which slots each of n new tokens sees."""
    m = np.zeros((n, base + n), dtype=bool)
    m[:, :base] = True
    for i in range(n):
        for j in range(n):
            m[i, base + j] = (j < 64 and (int(mask[i]) >> j) & 1 == 1) if mask is not None else j <= i
    return m


def attend(pages: Pages, q: np.ndarray, q_start, base, scale: float, visible=None, lse_in=None):
    """Per sequence and kv head: out [T, Hq, D], lse [T, Hq], mass {(s, h): [slots]} in 64 bits, with bounds of the
    errors that the kernels' roundings can make: out_tol, lse_tol, mass_tol of the same shapes.

    Roundings counted: scores are D/16 products of 16 terms accumulated in fp32, two roundings each (2^-23 of
    scale * sum|q| * 15 ks); the row sum of q, its product with kz and three more fp32 operations (16 * 2^-24 of scale * sum|q| *
    (15 ks + |kz|)); exponentials and their arguments 2^-20; a probability as fp16, 2^-11 of its part of the sum
    over codes; accumulation of the output 2^-16 of the terms' magnitudes; the output as bf16, 2^-8."""
    T, Hq, D = q.shape
    q = q.astype(np.float64)
    Hkv = pages.raw.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    out_tol, lse_tol = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    mass, mass_tol = {}, {}
    for s in range(len(base)):
        a, n, b = int(q_start[s]), int(q_start[s + 1] - q_start[s]), int(base[s])
        m = seen(b, n, None if visible is None else visible[a:a + n])
        m &= pages.valid(s, b + n)[None]
        for h in range(Hkv):
            kc, ks, kz = pages.entries(s, h, b + n, 0)
            vc, vs, vz = pages.entries(s, h, b + n, 1)
            any_row = m.any(0)
            with np.errstate(invalid="ignore"):
                kv = np.where(any_row[:, None], kz[:, None] + ks[:, None] * kc, 0.0)
            mass[s, h], mass_tol[s, h] = np.zeros(b + n), np.zeros(b + n)
            for i in range(n):
                see = m[i]
                if not see.any():
                    continue
                for x in range(G):
                    row = q[a + i, h * G + x]
                    S = scale * (kv[see] @ row)
                    top = S.max()
                    w = np.exp(S - top)
                    tot = w.sum()
                    p = w / tot
                    L = top + np.log(tot)
                    M = abs(scale) * np.abs(row).sum() * (15 * np.abs(ks[see]) + np.abs(kz[see]))
                    dS = (D / 16 * 2 * 2.0 ** -23 + 16 * 2.0 ** -24) * M + 2.0 ** -20 + 2.0 ** -22 * np.abs(S)
                    v = vz[see, None] + vs[see, None] * vc[see]
                    o = p @ v
                    out[a + i, h * G + x], lse[a + i, h * G + x] = o, L
                    lse_tol[a + i, h * G + x] = p @ dS + 2.0 ** -20 + 2.0 ** -22 * abs(L)
                    dp = p * (dS + p @ dS)
                    out_tol[a + i, h * G + x] = (2.0 ** -8 * np.abs(o) + dp @ np.abs(v - o)
                                                 + (2.0 ** -11 + 2.0 ** -16) * (p @ (vs[see, None] * vc[see]))
                                                 + 2.0 ** -16 * (p @ np.abs(vz[see])))
                    if lse_in is not None:
                        li = float(lse_in[a + i, h * G + x])
                        wt = np.exp(S - li)
                        mass[s, h][see] += wt
                        mass_tol[s, h][see] += wt * (dS + 2.0 ** -20 + 2.0 ** -22 * abs(li))
            mass_tol[s, h] += n * G * 2.0 ** -24 * mass[s, h]
    return out, lse, mass, out_tol, lse_tol, mass_tol


def evict(mass_row: np.ndarray, n: int, keep: int, recent: int) -> np.ndarray:
    """Kept old slots, ascending, of one (sequence, head) with n slots."""
    if n <= keep:
        return np.arange(n)
    free = n - recent
    m = mass_row[:free].astype(np.float64)
    order = np.lexsort((np.arange(free), -np.where(np.isnan(m), -np.inf, m), np.isnan(m)))
    return np.concatenate([np.sort(order[:keep - recent]), np.arange(free, n)]).astype(np.int64)
