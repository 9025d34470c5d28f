"""CPU oracle of the paged 8-bit cache: appending with rotation, and attention over it (float64 numpy).

Test infrastructure only.  A cache is codes uint8 [n_pages, n_kv, P, D] and scale bytes uint8
[n_pages, n_kv]; a batch is a list of (first row, new rows, length with them) and a page table.
"""
from __future__ import annotations

import numpy as np

from . import fp8_oracle as F


def rotate(x: np.ndarray, cos_sin: np.ndarray, style: str) -> np.ndarray:
    """x [T, heads, D], cos_sin [T, rot] (cosines, then sines): the pairs turned, the rest as it is."""
    y = np.array(x, dtype=np.float64)
    half = cos_sin.shape[1] // 2
    i = np.arange(half)
    a, b = (i, i + half) if style == "half" else (2 * i, 2 * i + 1)
    c, s = cos_sin[:, None, :half], cos_sin[:, None, half:]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def scale_byte(amax: np.ndarray) -> np.ndarray:
    """As the 8-bit format's, but for a group of zeros the least byte, so that it never raises a page's."""
    return np.where(np.asarray(amax) == 0, 0, F.scale_byte(amax)).astype(np.uint8)


def append(codes: np.ndarray, scales: np.ndarray, x: np.ndarray, seqs, table: np.ndarray) -> None:
    """x [T, n_kv, D]: every sequence's new rows into its pages, page by page (in place)."""
    P = codes.shape[2]
    for s, (a, n, length) in enumerate(seqs):
        j = length - n
        while j < length:
            page, lo = int(table[s, j // P]), j % P
            m = min(P - lo, length - j)
            new = x[a:a + m].transpose(1, 0, 2)                                   # [n_kv, m, D]
            byte = scale_byte(np.abs(new).max(axis=(1, 2)))
            if lo:
                byte = np.maximum(byte, scales[page])
                old = F.e4m3_to_f64(codes[page, :, :lo])
                with np.errstate(invalid="ignore"):
                    moved = old * (F.scale_value(scales[page]) / F.scale_value(byte))[:, None, None]
                grew = byte > scales[page]
                codes[page, grew, :lo] = F.f64_to_e4m3(moved[grew])
            scales[page] = byte
            with np.errstate(invalid="ignore"):
                codes[page, :, lo:lo + m] = F.f64_to_e4m3(new / F.scale_value(byte)[:, None, None])
            a, j = a + m, j + m


def values(codes: np.ndarray, scales: np.ndarray, table_row: np.ndarray, length: int) -> np.ndarray:
    """[n_kv, length, D]: the keys or values of one sequence."""
    P = codes.shape[2]
    pages = np.asarray(table_row[:-(-length // P)], dtype=np.int64)
    v = F.e4m3_to_f64(codes[pages]) * F.scale_value(scales[pages])[:, :, None, None]
    return v.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :length]


def seen(n: int, length: int, causal: bool = True, window: int = 0) -> np.ndarray:
    """[n, length]: which keys each new row sees."""
    pos = np.arange(length - n, length)[:, None]
    key = np.arange(length)[None, :]
    see = np.ones((n, length), dtype=bool)
    if causal:
        see &= key <= pos
    if window:
        see &= key > pos - window
    return see


def attention(q: np.ndarray, K: np.ndarray, V: np.ndarray, scale: float, see: np.ndarray):
    """q [n, heads, D] over K, V [n_kv, length, D]: (out [n, heads, D], weights [heads, n, length])."""
    n, heads, D = q.shape
    group = heads // K.shape[0]
    out = np.zeros((n, heads, D))
    weights = np.zeros((heads, n, K.shape[1]))
    for h in range(heads):
        with np.errstate(invalid="ignore"):
            x = np.where(see, (q[:, h] @ K[h // group].T) * scale, -np.inf)
            top = x.max(axis=1, keepdims=True, initial=-np.inf)
            p = np.exp(x - np.where(np.isfinite(top), top, 0.0))
            total = p.sum(axis=1, keepdims=True)
        weights[h] = np.divide(p, total, out=np.zeros_like(p), where=total != 0)
        with np.errstate(invalid="ignore"):
            out[:, h] = np.where(see.any(axis=1)[:, None], _weigh(weights[h], V[h // group], see), 0.0)
    return out, weights


def _weigh(w: np.ndarray, v: np.ndarray, see: np.ndarray) -> np.ndarray:
    """w @ v, where what a row does not see has no part in it (a NaN among it)."""
    if np.isfinite(v).all():
        return w @ v
    return np.stack([w[i, see[i]] @ v[see[i]] if see[i].any() else np.zeros(v.shape[1]) for i in range(len(w))])
