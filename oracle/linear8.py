"""Plain NumPy oracle of linear layers in 8 bits.

TEST INFRASTRUCTURE ONLY (imported by tests/).  Nothing is shared with the HIP library.

    a block is 128 consecutive values of a row (tall = 1) or 128 x 128 values (tall = 128)
    scale = 2^(s - 127), the smallest power of two with top / scale <= 448, s >= 10; top: the block's largest finite |value|
    code = value / scale, to the nearest e4m3 value, halves to even; NaN and infinity: the NaN code
    y = a b^T;  dW = grad^T x;  du = grad act'(u)
"""

from __future__ import annotations

import math

import numpy as np

from oracle.adamw8 import code_values

BLOCK, LOW = 128, 10


def _blocked(x, tall):
    rows, cols = x.shape
    out = np.zeros((-(-rows // tall) * tall, -(-cols // BLOCK) * BLOCK), dtype=x.dtype)
    out[:rows, :cols] = x
    return out.reshape(-1, tall, out.shape[1] // BLOCK, BLOCK)


def scales(x, tall: int = 1):
    """The scales' bytes, [rows / tall, blocks]."""
    mag = np.abs(_blocked(np.asarray(x, dtype=np.float64), tall))
    top = np.where(np.isfinite(mag), mag, 0.0).max(axis=(1, 3))
    out = np.empty(top.shape, dtype=np.uint8)
    for i, t in np.ndenumerate(top):
        p = LOW - 127
        while t > 448 * 2.0 ** p:
            p += 1
        out[i] = p + 127
    return out


def encode(x, tall: int = 1):
    """(codes [rows, cols], bytes [rows / tall, blocks]) as uint8, of values given in any float type."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    byte = scales(x, tall)
    y = _blocked(x, tall) / 2.0 ** (byte.astype(np.float64) - 127)[:, None, :, None]
    table = code_values().astype(np.float64)[:127]          # 0 .. 448, ascending
    with np.errstate(all="ignore"):
        mag = np.where(np.isfinite(y), np.abs(y), 0.0)
    hi = np.clip(np.searchsorted(table, mag), 1, 126)
    lo = hi - 1
    below, above = mag - table[lo], table[hi] - mag
    code = np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isfinite(y), code, 127) | (np.signbit(y) * 0x80)
    return code.astype(np.uint8).reshape(-1, code.shape[2] * BLOCK)[:rows, :cols], byte


def decode(codes, byte, tall: int = 1):
    rows, cols = codes.shape
    v = _blocked(code_values().astype(np.float64)[codes], tall) * 2.0 ** (byte.astype(np.float64) - 127)[:, None, :, None]
    return v.reshape(-1, v.shape[2] * BLOCK)[:rows, :cols]


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(u, kind: str):
    u = np.asarray(u, dtype=np.float64)
    if kind == "relu2":
        return np.where(u > 0, u * u, u * 0)
    if kind == "silu":
        return u / (1 + np.exp(-u))
    return u * 0.5 * _erfc(-u / math.sqrt(2.0)) if kind == "gelu" else u


def slope(u, kind: str):
    """(act'(u), the sum of its terms' magnitudes)."""
    u = np.asarray(u, dtype=np.float64)
    if kind == "relu2":
        s = 2 * np.maximum(u, 0)
        return s, np.abs(s)
    if kind == "silu":
        s = 1 / (1 + np.exp(-u))
        return s * (1 + u * (1 - s)), s * (1 + np.abs(u) * (1 - s))
    f, g = 0.5 * _erfc(-u / math.sqrt(2.0)), u * np.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    return f + g, f + np.abs(g)
