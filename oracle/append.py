"""64-bit definitions of the rotary KV append and of the 8-bit cache (numpy, plain loops).

Shares no code with the CUDA path. Cache bytes are carried as uint8 arrays.
"""
from __future__ import annotations

import numpy as np

MIN_EXP, MAX_EXP = -117, 119


def e4m3_values() -> np.ndarray:
    """The value of every e4m3 byte (S.1111.111 is NaN, no infinities)."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = -v if b & 128 else v
    out[0x7F] = out[0xFF] = np.nan
    return out


VALUES = e4m3_values()


def to_byte(y: float) -> int:
    """Nearest e4m3 byte, ties to the even mantissa, saturating; NaN and infinities give NaN."""
    if not np.isfinite(y):
        return 0x7F
    sign = 128 if np.signbit(y) else 0
    a = min(abs(float(y)), 448.0)
    e = max(int(np.floor(np.log2(a))), -6) if a > 0 else -6
    n = int(np.rint(a / 2.0 ** (e - 3)))          # rint rounds ties to even
    if n >= 16:
        n, e = n // 2, e + 1
    return sign | (n if n < 8 else ((e + 7) << 3) | (n - 8))


def half_step(y):
    """Half the distance between the e4m3 numbers around y."""
    a = np.clip(np.abs(y), 2.0 ** -6, 448.0)
    return 2.0 ** (np.floor(np.log2(a)) - 4)


def need(amax: float) -> int:
    x = MIN_EXP
    while x < MAX_EXP and amax > 448.0 * 2.0 ** x:
        x += 1
    return x


def rotate(x, positions, table, interleaved):
    """x [T, H, d] float64, table [positions, rot] -> rotated copy (rows with positions out of range unchanged)."""
    out = np.array(x, np.float64)
    if table is None:
        return out
    rot = table.shape[1]
    for t, pos in enumerate(positions):
        if not 0 <= pos < table.shape[0]:
            continue
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = float(table[pos, i]), float(table[pos, rot // 2 + i])
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return out


def append_q8(x, slots, cache, scale):
    """Put x [T, H, d] (float64) into cache [pages, H, P, d] / scale [pages, H, P / SB] (uint8), in place.

    Slots < 0 or past the cache are skipped. Returns {(page, head, place): x / 2^exponent before rounding}."""
    pages, heads, P, d = cache.shape
    sb = min(16, P)
    wanted = {}
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if not 0 <= s < pages * P:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and int(slots[t + n]) > int(slots[t + n - 1]) and int(slots[t + n]) // sb == s // sb:
            n += 1
        page, blk, offs = s // P, s % P // sb, [int(z) % P for z in slots[t:t + n]]
        for h in range(heads):
            run = x[t:t + n, h]
            fin = np.abs(run[np.isfinite(run)])
            e = need(float(fin.max()) if fin.size else 0.0)
            if offs[0] % sb != 0:
                was = int(scale[page, h, blk]) - 127
                if e > was:
                    for o in range(blk * sb, blk * sb + sb):
                        if o not in offs:
                            cache[page, h, o] = [to_byte(VALUES[b] * 2.0 ** (was - e)) for b in cache[page, h, o]]
                e = max(e, was)
            scale[page, h, blk] = e + 127
            for i, o in enumerate(offs):
                y = run[i] * 2.0 ** -e
                cache[page, h, o] = [to_byte(v) for v in y]
                wanted[(page, h, o)] = y
        t += n
    return wanted


def values(cache, scale):
    """What an 8-bit cache holds: [pages, H, P, d] float64."""
    sb = cache.shape[2] // scale.shape[2]
    return VALUES[cache] * np.repeat(2.0 ** (scale.astype(np.float64) - 127), sb, axis=2)[..., None]
