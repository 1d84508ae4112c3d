"""The 8-bit latent cache by its definition, fp64 (oracle, test infrastructure only).

A group of 32 values shares a scale 2^e, e the least exponent in [-110, 119] with
max |c| / 2^e <= 448 (119 where none is: such a value becomes 448); a value is the e4m3 number (sign, 4 exponent bits of bias 7, 3
fraction bits, no infinities) nearest to c / 2^e, ties to the even code. A group with a
non-finite value is NaN throughout (scale byte 255).
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 32


def e4m3_values() -> np.ndarray:
    """The magnitudes of codes 0 .. 126."""
    out = []
    for code in range(127):
        e, f = code >> 3, code & 7
        out.append(math.ldexp(f / 8, -6) if e == 0 else math.ldexp(1 + f / 8, e - 7))
    return np.array(out)


def nearest_code(x: np.ndarray) -> np.ndarray:
    """e4m3 code of each value (|x| <= 448)."""
    v = e4m3_values()
    a = np.abs(x)
    hi = np.clip(np.searchsorted(v, a), 1, 126)
    lo = hi - 1
    up, down = v[hi] - a, a - v[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(a == 0, 0, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def encode(c: np.ndarray):
    """c [n, r] -> codes [n, r] uint8, scale bytes [n, r / 32] uint8."""
    c = np.asarray(c, np.float64)
    g = c.reshape(c.shape[0], -1, GROUP)
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], g, 0.0)
    top = np.abs(g).max(-1)
    # top = f 2^k with f in [1/2, 1): 448 2^(k - 9) = 0.875 2^k is enough for f <= 0.875
    f, k = np.frexp(top)
    e = np.where(top > 0, np.clip(k - 9 + (f > 0.875), -110, 119), -110).astype(np.int64)
    codes = nearest_code(np.clip(np.ldexp(g, -e[..., None]), -448, 448))
    codes[~finite] = 0x7F
    return codes.reshape(c.shape), np.where(finite, e + 127, 255).astype(np.uint8)


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What codes [n, r] and scale bytes [n, r / 32] stand for."""
    v = np.append(e4m3_values(), np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, GROUP, axis=1)
