"""Log probabilities, entropy and the likeliest ids of rows of logits in fp64
(test infrastructure only).

NaN counts as -infinity.  Where a row holds +infinity those ids share the
probability equally; a row of -infinity only gives -infinity for every id and
entropy 0.  Ranking is by (logit descending, id ascending) on the given values.
"""
from __future__ import annotations

import numpy as np


def row(x) -> tuple[np.ndarray, float]:
    """(log probability of every id, entropy in nats) of one row."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64))
    m = x.max()
    if m == -np.inf:
        return np.full(x.shape, -np.inf), 0.0
    if m == np.inf:
        n = int((x == np.inf).sum())
        return np.where(x == np.inf, -np.log(n), -np.inf), float(np.log(n))
    lp = (x - m) - np.log(np.exp(x - m).sum())
    p = np.exp(lp)
    return lp, float(-(p[p > 0] * lp[p > 0]).sum())


def top(x, k: int) -> np.ndarray:
    """The k likeliest ids of one row."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64))
    return np.lexsort((np.arange(x.size), -x))[:k]
