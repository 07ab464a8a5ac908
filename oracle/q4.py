"""64-bit definitions of head norms and of the 4-bit cache (numpy, plain loops and tables).

Shares no code with the CUDA path. A number of the cache is code * scale: e2m1 codes, two to
a byte (even column in the low half), one scale byte for every 16 columns.
"""
from __future__ import annotations

import numpy as np

GROUP = 16
CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIN_SCALE, MAX_SCALE, NAN_SCALE = 1, 0xE2, 255           # bytes the writer produces: 2^-17, 10240, and NaN


def scale_values() -> np.ndarray:
    """The number every scale byte stands for: 5 bits of exponent, 3 of mantissa."""
    out = np.empty(256)
    for b in range(256):
        e, m = b >> 3, b & 7
        out[b] = m * 2.0 ** -17 if e == 0 else (8 + m) * 2.0 ** (e - 18)
    out[248:] = np.nan
    out[248] = np.inf
    return out


SCALES = scale_values()


def nearest(x: float, table) -> int:
    """Index of the number of `table` (ascending) nearest to x, ties to the even index, clamped to the ends."""
    i = int(np.searchsorted(table, x))
    if i == 0 or i == len(table):
        return min(i, len(table) - 1)
    lo, hi = x - table[i - 1], table[i] - x
    return i - 1 if lo < hi or (lo == hi and (i - 1) % 2 == 0) else i


def to_scale(amax: float) -> int:
    """The scale byte of a group whose largest magnitude is amax."""
    if not np.isfinite(amax):
        return NAN_SCALE
    return min(max(nearest(amax / 6.0, SCALES[:248]), MIN_SCALE), MAX_SCALE)


def to_code(y: float) -> int:
    return nearest(abs(y), CODES) + (8 if y < 0 else 0)


def quantised(x):
    """x [..., d] float64 -> (code per column [..., d], scale byte per group [..., d / 16]); the codes of NaN groups are 0."""
    flat = x.reshape(-1, GROUP)
    code, scale = np.zeros(flat.shape, np.uint8), np.zeros(len(flat), np.uint8)
    for i, g in enumerate(flat):
        scale[i] = to_scale(np.abs(g).max())
        if scale[i] != NAN_SCALE:
            code[i] = [to_code(v / SCALES[scale[i]]) for v in g]
    return code.reshape(x.shape), scale.reshape(*x.shape[:-1], x.shape[-1] // GROUP)


def packed(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def unpacked(cache):
    out = np.empty((*cache.shape[:-1], 2 * cache.shape[-1]), np.uint8)
    out[..., 0::2], out[..., 1::2] = cache & 15, cache >> 4
    return out


def values(cache, scale):
    """What a 4-bit cache holds, float64 [..., d]."""
    code = unpacked(cache)
    x = np.where(code & 8, -1.0, 1.0) * CODES[code & 7]
    with np.errstate(invalid="ignore"):
        return x * np.repeat(SCALES[scale], GROUP, axis=-1)


def head_norm(x, weight, eps):
    """x [T, H, d] float64: every head to unit mean square (eps beside it), times weight [d]."""
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
