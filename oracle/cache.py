"""Appending rows to a KV cache with rotation, and attention over a cache, in
fp64 numpy from their definitions.  A cache here is a list of per-sequence
arrays [Hkv, len, dh]; layouts (pages, codes and scales) are unpacked by the
caller."""
from __future__ import annotations

import numpy as np

from .block import rope

E4M3_MAX = 448.0
E4M3_SCALE_EXP = (-24, 60)


def rotated(x: np.ndarray, start: int, base: float) -> np.ndarray:
    """Rows x [n, heads, dh] turned at positions start, start + 1, ..."""
    return rope(x, range(start, start + len(x)), base)


def visible(pos: int, length: int, window: int = 0, sinks: int = 0) -> np.ndarray:
    """Which of `length` keys the query at position `pos` sees."""
    j = np.arange(length)
    see = j <= pos
    if window > 0:
        see &= (j > pos - window) | (j < sinks)
    return see


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, first: int, window: int = 0, sinks: int = 0,
           scale: float | None = None):
    """Queries q [m, H, dh] at positions first.. over k, v [Hkv, len, dh]: the
    outputs [m, H, dh], the weighted magnitudes sum_j w_j |v_j| of the same shape
    and the largest sum_d |q_d k_d| * scale per (query, head)."""
    m, H, dh = q.shape
    Hkv, L, _ = k.shape
    scale = 1 / np.sqrt(dh) if scale is None else scale
    out, mag, top = np.zeros((m, H, dh)), np.zeros((m, H, dh)), np.zeros((m, H))
    for i in range(m):
        see = visible(first + i, L, window, sinks)
        if not see.any():
            continue
        for h in range(H):
            kk, vv = k[h // (H // Hkv)][see], v[h // (H // Hkv)][see]
            z = kk @ q[i, h] * scale
            w = np.exp(z - z.max())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
            top[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, mag, top


def e4m3_scale(top: float) -> float:
    """The block scale for a largest finite magnitude `top`."""
    lo, hi = E4M3_SCALE_EXP
    if top == 0:
        return 2.0 ** lo
    e = int(np.ceil(np.log2(top / E4M3_MAX)))
    return 2.0 ** min(max(e, lo), hi)
