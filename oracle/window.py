"""Attention over a sliding window with sinks, unsplit, in fp64 (test
infrastructure only): the row at position p sees key j <= p if j > p - window or
j < sinks; window 0 means every key j <= p.  A row that sees nothing (a sequence
of length 0) gives zeros.
"""
from __future__ import annotations

import math

import numpy as np


def visible(p: int, n: int, window: int, sinks: int) -> np.ndarray:
    """Whether the row at position p sees key j, j < n."""
    return np.array([j <= p and (window == 0 or p - j < window or j < sinks) for j in range(n)], dtype=bool)


def row(q: np.ndarray, k: np.ndarray, v: np.ndarray, p: int, window: int, sinks: int, scale=None) -> np.ndarray:
    """fp64 q [Hq][D], k and v [slots][Hkv][D] -> fp64 [Hq][D] for the row at position p."""
    hq, d = q.shape
    group = hq // k.shape[1]
    at = np.nonzero(visible(p, p + 1, window, sinks))[0] if p >= 0 else np.zeros(0, dtype=int)
    out = np.zeros((hq, d))
    if len(at) == 0:
        return out
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    for h in range(hq):
        s = k[at, h // group] @ q[h] * scale
        w = np.exp(s - s.max())
        out[h] = (w / w.sum()) @ v[at, h // group]
    return out
