"""Trees of drafted tokens behind a cached context (test infrastructure only).

Sequence b has ``ctx[b]`` cached keys and ``n[b]`` drafted nodes; ``parent[i]``
is the node's parent (below i) or -1.  A node with t ancestors is the token at
position ctx + t; its keys and values sit in cache slot ctx + i, and it sees the
context, its ancestors and itself.  So a node is the decode row of length
ctx + t + 1 over the context followed by its path, which is how ``attention``
computes it: the path's slots are gathered and the plain decode of that length
is taken.
"""
from __future__ import annotations

import numpy as np

from . import attention as _attention


def path_of(parent, i: int) -> list[int]:
    """The node's ancestors and itself, the oldest first."""
    path = []
    while i >= 0:
        path.append(i)
        if parent[i] >= i:
            raise ValueError("a parent's index must be below its child's")
        i = int(parent[i])
    return path[::-1]


def valid(parent, n: int) -> bool:
    return all(-1 <= int(parent[i]) < i for i in range(n))


def attention(q_bits, k_bits, v_bits, ctx: int, parent, scale=None):
    """One sequence: q [n][Hq][D], caches [slots][Hkv][D] -> bf16 [n][Hq][D]."""
    out = []
    for i in range(q_bits.shape[0]):
        slots = np.array(list(range(ctx)) + [ctx + j for j in path_of(parent, i)])
        out.append(_attention.decode(q_bits[i: i + 1], k_bits[slots][None], v_bits[slots][None], [len(slots)],
                                     scale)[0])
    return np.stack(out)


def positions(ctx: int, parent) -> np.ndarray:
    return np.array([ctx + len(path_of(parent, i)) - 1 for i in range(len(parent))])


def accept(parent, tokens, next_tokens) -> list[int]:
    """The nodes taken: node 0, then the lowest child that holds the token the
    model put after the last one taken."""
    if len(parent) == 0:
        return []
    path = [0]
    while True:
        nxt = [j for j in range(len(parent)) if parent[j] == path[-1] and tokens[j] == next_tokens[path[-1]]]
        if not nxt:
            return path
        path.append(nxt[0])
