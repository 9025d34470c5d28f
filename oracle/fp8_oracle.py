"""CPU oracle of the block-scaled 8-bit format, its projections and the residual norm (float64 numpy).

Test infrastructure only, like the rest of this package.  The format: e4m3 codes (1 sign, 4
exponent, 3 mantissa bits, bias 7; no infinity, 0x7F and 0xFF are NaN, largest value 448) with one
power-of-two scale per group of 128, held as the byte e + 127 (255 is NaN).
"""
from __future__ import annotations

import numpy as np

from .tp_oracle import apply_act

GROUP = 128
E4M3_MAX = 448.0


def _code_value(code: int) -> float:
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))


VALUES = np.array([_code_value(c) for c in range(256)])
_POSITIVE = VALUES[:127]    # ascending


def e4m3_to_f64(codes: np.ndarray) -> np.ndarray:
    return VALUES[np.asarray(codes, dtype=np.uint8)]


def f64_to_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest code (ties to the even one) of values within +-448; NaN becomes 0x7F."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), E4M3_MAX)
    hi = np.clip(np.searchsorted(_POSITIVE, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(_POSITIVE[hi] == a, hi, code) | np.where(np.signbit(v), 0x80, 0)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def scale_byte(amax: np.ndarray) -> np.ndarray:
    """e + 127 for the least e with amax <= 448 * 2^e, clamped; 127 for zero, 255 for NaN and infinity."""
    amax = np.asarray(amax, dtype=np.float64)
    finite = np.isfinite(amax)
    m, k = np.frexp(np.where(finite, amax, 1.0))          # amax = m 2^k, m in [0.5, 1); 448 = 0.875 * 2^9
    e = np.clip(np.where(m > 0.875, k - 8, k - 9), -127, 127)
    return np.where(~finite, 255, np.where(amax == 0, 127, e + 127)).astype(np.uint8)


def scale_value(byte: np.ndarray) -> np.ndarray:
    b = np.asarray(byte, dtype=np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def spread(scales: np.ndarray, shape, block_rows: int) -> np.ndarray:
    """A scale for every element of a [rows, cols] matrix."""
    return np.repeat(np.repeat(scales, block_rows, 0)[:shape[0]], GROUP, 1)[:, :shape[1]]


def group_amax(x: np.ndarray, block_rows: int) -> np.ndarray:
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // GROUP)
    pad = np.zeros((nr * block_rows, nc * GROUP))
    pad[:rows, :cols] = np.abs(x)
    return pad.reshape(nr, block_rows, nc, GROUP).max(axis=(1, 3))


def quantize(x: np.ndarray, block_rows: int):
    """(codes, scale bytes) of float64 values."""
    byte = scale_byte(group_amax(x, block_rows))
    with np.errstate(invalid="ignore"):
        return f64_to_e4m3(x / spread(scale_value(byte), x.shape, block_rows)), byte


def dequantize(codes: np.ndarray, byte: np.ndarray, block_rows: int) -> np.ndarray:
    return e4m3_to_f64(codes) * spread(scale_value(byte), codes.shape, block_rows)


def linear_terms(x: np.ndarray, w: np.ndarray):
    """(X . W^T, the sum of the products' magnitudes)."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def colwise(x: np.ndarray, w: np.ndarray, bias=None, act: str = "none") -> np.ndarray:
    y = x @ w.T
    return apply_act(y if bias is None else y + bias, act)


def normalise(v: np.ndarray, kind: str, eps: float, weight=None, bias=None) -> np.ndarray:
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    v = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    v = v if weight is None else v * weight
    return v if bias is None else v + bias


def residual_norm(x, y=None, *, norm="none", weight=None, bias=None, scale=None, shift=None, post_norm="none",
                  post_weight=None, post_bias=None, gate=None, alpha=1.0, eps=1e-6, rows_per_mod=1):
    """(h, u) in float64; gate, scale and shift are [mod_rows, D] tables."""
    row = np.arange(x.shape[0]) // rows_per_mod
    h = alpha * x
    if y is not None:
        b = normalise(y, post_norm, eps, post_weight, post_bias)
        h = h + (b if gate is None else gate[row] * b)
    u = normalise(h, norm, eps, weight, bias)
    if scale is not None:
        u = u * (1 + scale[row])
    if shift is not None:
        u = u + shift[row]
    return h, u
