"""Microscaled 4 bits in double precision (numpy), from the definitions in
include/sampler.h: codes and scales of a matrix, its values, and the LM head's
product. Plain loops over blocks; nothing is shared with the CUDA path."""
from __future__ import annotations

import numpy as np

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
LEAST = 2.0 ** -100


def nearest(x, digits, least):
    """The nearest number of so many significant bits whose exponent is `least` or more; ties to even."""
    _, e = np.frexp(np.maximum(np.abs(x), 2.0 ** least))
    step = 2.0 ** (e - digits).astype(np.float64)
    return np.round(x / step) * step


def least_power(x):
    """The exponent of the least power of two that is x or more (x > 0)."""
    f, e = np.frexp(x)
    return e - (f == 0.5)


def e4m3_code(x):
    """The e4m3 code of a number that e4m3 has, 0 or more."""
    if x < 2.0 ** -6:
        return int(x * 2.0 ** 9)
    f, e = np.frexp(x)  # f in [0.5, 1)
    return int((e + 6) * 8 + (f * 16 - 8))


def e4m3_value(code):
    e, m = int(code) >> 3 & 15, int(code) & 7
    if int(code) & 0x7f == 0x7f:
        return np.nan
    return (1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9


def scale_value(code, block):
    if block == 16:
        return e4m3_value(code)
    return np.nan if code == 0xff else 2.0 ** (int(code) - 127)


def scale_place(rows, cols, block):
    """[rows, blocks] places of the scales' bytes, and the size of all."""
    blocks = -(-cols // block)
    tiles = -(-blocks // 4)
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None]
    return ((r // 128) * tiles + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4, -(-rows // 128) * tiles * 512


def quantize(x, block):
    """(packed codes [rows, cols / 2 rounded up], scales as they lie, row scales, values in double)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    place, size = scale_place(rows, cols, block)
    scales, row_scale = np.zeros(size, np.uint8), np.ones(rows, np.float32)
    codes, values = np.zeros((rows, cols + cols % 2), np.uint8), np.zeros((rows, cols))
    for r in range(rows):
        starts = range(0, cols, block)
        most = [np.abs(x[r, b:b + block]).max() for b in starts]
        if block == 16:
            finite = [m for m in most if np.isfinite(m)]
            row_scale[r] = 2.0 ** float(least_power(max([LEAST] + finite) / 2688.0))
        for j, b in enumerate(starts):
            v = x[r, b:b + block]
            if not np.isfinite(most[j]):
                scales[place[r, j]] = 0x7f if block == 16 else 0xff
                values[r, b:b + block] = np.nan
                continue
            if block == 16:
                s = float(nearest(most[j] / 6.0 / float(row_scale[r]), 4, -6))
                scales[place[r, j]] = e4m3_code(s)
            else:
                e = max(int(least_power(max(most[j], 2.0 ** -200) / 6.0)), -127)
                s = 2.0 ** e
                scales[place[r, j]] = e + 127
            unit = s * float(row_scale[r])
            q = np.minimum(np.abs(nearest(v / unit, 2, 0)), 6.0) if unit > 0 else np.zeros_like(v)
            c = np.searchsorted(CODES, q)
            codes[r, b:b + len(v)] = c + 8 * np.signbit(v)
            values[r, b:b + block] = np.copysign(q, v) * unit
    return codes[:, 0::2] | codes[:, 1::2] << 4, scales, row_scale, values


def values(packed, scales, row_scale, cols, block):
    """The numbers that codes and scales stand for, in double."""
    rows = packed.shape[0]
    c = np.empty((rows, 2 * packed.shape[1]), np.uint8)
    c[:, 0::2], c[:, 1::2] = packed & 15, packed >> 4
    c = c[:, :cols]
    x = np.where(c > 7, -1.0, 1.0) * CODES[c & 7]
    place, _ = scale_place(rows, cols, block)
    table = np.array([scale_value(k, block) for k in range(256)])
    s = table[scales[place]]
    if row_scale is not None:
        s = s * np.asarray(row_scale, np.float64)[:, None]
    return x * np.repeat(s, block, 1)[:, :cols]


def head(hidden, weight):
    """(logits, the sum of the products' magnitudes) of two operands' values in double."""
    return hidden @ weight.T, np.abs(hidden) @ np.abs(weight).T
