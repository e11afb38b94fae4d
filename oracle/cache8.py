"""The 8-bit key/value cache's codes, in fp64 (test infrastructure only).

A vector of D bf16 values x (one token, one kv head) is held as D codes and one
exponent E; element d stands for code[d] * 2^E.  With amax = max |x_d|:

    e4m3: E = min { e : amax <= 448 * 2^e }, clamped to [-100, 119]
    int8: E = min { e : amax <= 127 * 2^e }, clamped to [-100, 121]

and code = x * 2^-E rounded to the nearest code, ties to the code whose last
bit is 0, saturating at the largest code.  A vector that holds an infinity or a
NaN has E = -128 and codes 0, and stands for NaN.

e4m3 code s eeee mmm: (-1)^s * 2^(e - 7) * (1 + m/8), and 2^-6 * m/8 for e = 0
(0x7F and 0xFF would be NaN and are not used).  Written from these definitions
by search over the 127 magnitudes.
"""
from __future__ import annotations

import numpy as np

from . import bf16

LIMIT = {"e4m3": 448.0, "int8": 127.0}
MAX_EXP = {"e4m3": 119, "int8": 121}
MIN_EXP = -100
NAN_EXP = -128


def e4m3_magnitudes() -> np.ndarray:
    """Values of codes 0x00 .. 0x7E."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, 2.0 ** -6 * m / 8.0, 2.0 ** (e - 7.0) * (1 + m / 8.0))


def exponent(x: np.ndarray, fmt: str) -> np.ndarray:
    """x fp64 [..., D] -> E int [...]."""
    amax = np.abs(x).max(-1)
    out = np.full(amax.shape, MIN_EXP)
    for i, a in np.ndenumerate(amax):
        if not np.isfinite(a):
            out[i] = NAN_EXP
            continue
        e = MIN_EXP
        while e < MAX_EXP[fmt] and a > LIMIT[fmt] * 2.0 ** e:
            e += 1
        out[i] = e
    return out


def quantise(x_bits, fmt: str):
    """bf16 bits [..., D] -> (codes [..., D] as the raw bytes (uint8), exponents int8 [...])."""
    x = bf16.to_f64(x_bits)
    E = exponent(x, fmt)
    marked = E == NAN_EXP
    y = np.where(marked[..., None], 0.0, x) * 2.0 ** -np.where(marked, 0, E).astype(np.float64)[..., None]
    if fmt == "int8":
        codes = np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)   # np.rint: half to even
    else:
        mag = e4m3_magnitudes()
        a = np.minimum(np.abs(y), 448.0)
        hi = np.searchsorted(mag, a)                     # first magnitude >= a
        lo = np.maximum(hi - 1, 0)
        up, down = mag[hi] - a, a - mag[lo]
        pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        pick = np.where(hi == 0, 0, pick)
        codes = (pick | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)
    return codes, E.astype(np.int8)


def values(codes: np.ndarray, E: np.ndarray, fmt: str) -> np.ndarray:
    """Raw bytes [..., D] and exponents [...] -> fp64 values."""
    codes = np.asarray(codes, dtype=np.uint8)
    if fmt == "int8":
        c = codes.view(np.int8).astype(np.float64)
    else:
        c = e4m3_magnitudes()[codes & 0x7F] * np.where(codes & 0x80, -1.0, 1.0)
    E = np.asarray(E, dtype=np.int64)
    return np.where((E == NAN_EXP)[..., None], np.nan, c * 2.0 ** np.where(E == NAN_EXP, 0, E).astype(np.float64)[..., None])
