"""Plain NumPy oracle of AdamW with 8-bit states, in float32 with one rounding per operation.

TEST INFRASTRUCTURE ONLY (imported by tests/).  Nothing is shared with the HIP
library.  NumPy's float32 operations are the IEEE ones, so a correct kernel
gives these results bit for bit; the update itself is held against the
float64 AdamW of oracle/adamw.py.

A state is (codes, scale): e4m3 codes (uint8) and one float32 scale per 256
values; the first moment is value(code) * scale, the square root of the second
likewise.  Written back per block with top = the largest magnitude:
    scale = top * fl(1/448);  inverse = 448 * (1 / top)  (0 where top < 2^-100)
    y = |x| * inverse, to the nearest code below or above: the fp32 pattern of
    y * 2^-120, plus the dither, without its low 20 bits; at most 126
"""

from __future__ import annotations

import numpy as np

BLOCK = 256
F = np.float32


def code_values() -> np.ndarray:
    """The 256 values of the e4m3 codes (4 exponent bits, bias 7; no infinities, 0x7F is NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where(c & 0x80, -v, v)
    v[(c & 0x7F) == 0x7F] = np.nan
    return v.astype(F)


def _blocks(x: np.ndarray) -> np.ndarray:
    n = -(-len(x) // BLOCK)
    out = np.zeros(n * BLOCK, dtype=x.dtype)
    out[:len(x)] = x
    return out.reshape(n, BLOCK)


def decode(codes, scale) -> np.ndarray:
    return (code_values()[_blocks(codes)] * scale[:, None]).reshape(-1)[:len(codes)]


def encode(x, dither, keep_positive: bool):
    """(codes, scale) of float32 values; dither: per-value integers added to the 20 bits that are cut."""
    b = _blocks(x)
    mag = np.abs(b)
    with np.errstate(all="ignore"):
        top = mag.max(axis=1)
        scale = np.where(np.isfinite(top), top * F(1.0 / 448.0), F(np.nan)).astype(F)
        inverse = np.where(top >= F(2.0 ** -100), F(448.0) * (F(1.0) / top), F(0)).astype(F)
        y = (mag * inverse[:, None]) * F(2.0 ** -120)
    bits = (y.view(np.uint32) & 0x7FFFFFFF).astype(np.int64)
    code = np.minimum((bits + _blocks(dither)) >> 20, 126)
    if keep_positive:
        code = np.where((b > 0) & (code == 0), 1, code)
    else:
        code = code | (np.signbit(b) * 0x80)
    return code.astype(np.uint8).reshape(-1)[:len(x)], scale


def mix(x):
    x = np.asarray(x, dtype=np.uint64) & 0xFFFFFFFF
    x ^= x >> np.uint64(16)
    x = x * np.uint64(0x6A09E667) & np.uint64(0xFFFFFFFF)
    x ^= x >> np.uint64(15)
    x = x * np.uint64(0xBB67AE85) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def dithers(n: int, seed, step: int, place: int):
    """(for exp_avg, for rms) of n values."""
    if seed is None:
        d = np.full(n, 0x7FFFF, dtype=np.int64)
        return d, d
    seed = (seed & 0xFFFFFFFF) ^ int(mix(seed >> 32 & 0xFFFFFFFF))
    key = mix(mix((seed + 0x9E3779B9 * step) & 0xFFFFFFFF) + np.uint64(place))
    x = mix(key + np.arange(n, dtype=np.uint64)).astype(np.int64)
    return (x >> 16) << 4, (x & 0xFFFF) << 4


def step(p, g, state, *, lr, beta1, beta2, eps, wd, t, seed=None, place=0, ema=None, decay=0.0):
    """One step on float32 arrays; state: ((codes, scale), (codes, scale)) or (m, v).  Returns p', state', ema'."""
    lr, beta1, beta2, eps, wd, decay = (F(x) for x in (lr, beta1, beta2, eps, wd, decay))
    one = F(1)
    size = F(float(lr) / (1.0 - float(beta1) ** t))
    ibc2 = F(1.0 / np.sqrt(1.0 - float(beta2) ** t))
    q8 = isinstance(state[0], tuple)
    if q8:
        m = decode(*state[0])
        r = decode(*state[1])
        v = r * r
    else:
        m, v = state
    with np.errstate(all="ignore"):
        m = m * beta1 + g * (one - beta1)
        v = v * beta2 + (g * g) * (one - beta2)
        root = np.sqrt(v)
        p = p * (one - lr * wd) - (m / (root * ibc2 + eps)) * size
        if ema is not None:
            ema = ema * decay + p * (one - decay)
    if q8:
        dm, dr = dithers(len(p), seed, t, place)
        return p, (encode(m, dm, False), encode(root, dr, True)), ema
    return p, (m, v), ema
