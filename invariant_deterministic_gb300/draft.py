"""Decoding with drafted tokens: several tokens of a request per step, the same
tokens as decoding them one by one.

A drafter proposes a tree of continuations for each request (node 0 is the
token that was decided last, its descendants are guesses).  One step runs every
node of every tree through the model (Decoder.tree_layers), samples the model's
own token after each node with the request's settings, the history of the node's
path and the Philox counter of its position, and keeps the path on which the
guesses agree with those tokens (kinv.tree_accept), which also moves the path's
keys and values to their positions.  A node's logits have the bits of the decode
step at its place and the sampler depends on the row, the settings and the step
alone, so the tokens are those of run_requests whatever the drafter guesses; a
good guess only makes a step yield more of them.
"""
from __future__ import annotations

import numpy as np
import torch

from . import kinv, synth
from .model import Decoder


def ngram_tree(tokens, max_nodes: int, n: int = 2, depth: int = 8):
    """Guesses by lookup: wherever the last n (or fewer, down to one) tokens
    occurred before, what followed them, up to ``depth`` tokens; the latest
    occurrences first, merged into one tree of at most max_nodes nodes.
    Returns (node tokens, parents); node 0 is the last token itself."""
    tokens = list(tokens)
    nodes, parents, child = [tokens[-1]], [-1], {}
    for size in range(min(n, len(tokens) - 1), 0, -1):
        tail = tokens[-size:]
        for at in range(len(tokens) - size - 1, -1, -1):
            if len(nodes) >= max_nodes:
                return nodes, parents
            if tokens[at: at + size] != tail:
                continue
            cur = 0
            for t in tokens[at + size: at + size + depth]:
                if (cur, t) not in child:
                    if len(nodes) >= max_nodes:
                        break
                    child[(cur, t)] = len(nodes)
                    nodes.append(t)
                    parents.append(cur)
                cur = child[(cur, t)]
    return nodes, parents


class DraftDecoder:
    """Steps of drafted trees over a Decoder's slots.  The decoder's chunk
    buffers bound a step's nodes (max_batch * max_nodes rows at most), and each
    slot needs max_nodes cache positions behind its last token.  The workspace is
    that of max_batch trees of max_nodes nodes in the whole cache (for an 8B layer
    34 MB with 16 slots of 2,048 tokens and 16 nodes, 0.5 GB with 32,768 tokens).
    A step runs eagerly: 36 layers of 8B, 500 tokens, take 4.9 ms for one tree of
    8 nodes, 6.5 for 16 of 8 and 10.8 for 16 of 16, a captured decode step 2.9 for
    one request and 3.3 for 16."""

    def __init__(self, dec: Decoder, max_nodes: int = 16):
        if not 1 <= max_nodes <= kinv.TREE_MAX_NODES:
            raise ValueError(f"max_nodes must lie in 1..{kinv.TREE_MAX_NODES}")
        if dec.B * max_nodes > dec.max_rows:
            raise ValueError("the decoder's max_chunk must hold max_batch * max_nodes rows")
        if getattr(dec, "cache", "bf16") != "bf16" or getattr(dec.s, "window", 0):
            raise ValueError("drafted decoding needs a bf16 cache and attention without a window")
        self.dec, self.max_nodes = dec, max_nodes
        rows = dec.B * max_nodes
        i32 = dict(dtype=torch.int32, device=dec.dev)
        self.logits = torch.zeros(rows, dec.s.vocab, dtype=torch.float32, device=dec.dev)
        self.sampled = torch.zeros(rows, **i32)
        # for the widest step: every slot with max_nodes nodes, the whole cache
        seqs, most = torch.zeros(dec.B, **i32), torch.zeros(rows, **i32)
        widest = kinv.Tree(seqs, seqs, seqs, most, max_nodes, dec.Lmax)
        self.ws = torch.empty(max(16, kinv.attn_tree_workspace(widest, dec.s.n_q, dec.s.n_kv, dec.s.head_dim)),
                              dtype=torch.uint8, device=dec.dev)
        self.requests = []

    def start(self, prompts, params, chunk: int = 0) -> None:
        """Request i takes slot i: its prompt but for the last token is prefilled."""
        dec = self.dec
        if len(prompts) > dec.B:
            raise ValueError("more requests than the decoder's slots")
        for i, p in enumerate(prompts):
            if len(p) < 1 or len(p) > dec.Lmax:
                raise ValueError("prompt empty or too long for the decoder's cache")
            if len(p) > 1:
                dec.prefill(i, torch.tensor(list(p[:-1]), dtype=torch.int32, device=dec.dev), chunk=chunk)
        self.requests = [list(map(int, p)) for p in prompts]
        self.prompt_len = [len(p) for p in prompts]
        dec.set_sampling(params)

    def _inputs(self, trees):
        """Host arrays of a step: per node its token, parent, request, position
        in the request's output, and the sampler's history (its path included)."""
        dec, ld = self.dec, self.dec.hist_ld
        if len(trees) != len(self.requests):
            raise ValueError("a step has one tree per request (an empty one leaves its request as it is)")
        token, parent, owner, step, n, hist, hist_len = [], [], [], [], [], [], []
        for b, (nodes, parents) in enumerate(trees):
            seq = self.requests[b]
            if len(nodes) != len(parents) or len(nodes) > self.max_nodes:
                raise ValueError("a tree has one parent per node and at most max_nodes nodes")
            if len(nodes) == 0:
                n.append(0)
                continue
            if nodes[0] != seq[-1] or parents[0] != -1:
                raise ValueError("node 0 of a tree is the request's last token")
            if len(seq) - 1 + len(nodes) > dec.Lmax:
                raise ValueError("the tree does not fit behind the request in the decoder's cache")
            paths = []
            for i, (t, p) in enumerate(zip(nodes, parents)):
                if i and not 0 <= p < i:
                    raise ValueError("a node's parent comes before it")
                if not 0 <= t < dec.s.vocab:
                    raise ValueError("a drafted token lies outside the vocabulary")
                paths.append(paths[p] + [t] if i else [])
                tail = (seq[-ld:] + paths[i])[-ld:]
                token.append(t), parent.append(p), owner.append(b)
                step.append(len(seq) - self.prompt_len[b] + len(paths[i]))
                hist.append(tail + [0] * (ld - len(tail)))
                hist_len.append(len(tail))
            n.append(len(nodes))
        return token, parent, owner, step, n, hist, hist_len

    def step(self, trees):
        """One step with a tree per request, (tokens, parents) each (an empty
        one leaves its request as it is).  Returns the tokens each decided."""
        dec = self.dec
        token, parent, owner, step, n, hist, hist_len = self._inputs(trees)
        rows = len(token)
        if rows == 0:
            return [[] for _ in trees]
        up = lambda v, dt=torch.int32: torch.tensor(v, dtype=dt).to(dec.dev)
        ctx = [len(r) - 1 for r in self.requests]
        tree = kinv.Tree(up(ctx), up(n), up(np.cumsum([0] + n[:-1]).tolist()), up(parent), self.max_nodes, dec.Lmax)
        tokens = up(token)
        kinv.embed(dec.w["embed"], tokens, out=dec.x[:rows])
        dec.tree_layers(tree, rows, self.ws)
        logits = dec.lm_head(0, self.logits[:rows])
        size = synth.SAMPLING_DTYPE.itemsize
        params = dec.params.view(-1, size)[up(owner, torch.int64)].contiguous()
        sampled = kinv.sample(logits, params, up(hist), up(hist_len), up(step, torch.int64), out=self.sampled[:rows])
        count, _, out = kinv.tree_accept(tree, tokens, sampled, dec.kv)
        got = [row[:c] for row, c in zip(out.cpu().tolist(), count.cpu().tolist())]
        for r, t in zip(self.requests, got):
            r.extend(t)
        return got


def run_requests_drafted(dec: Decoder, prompts, params, steps: int, draft=ngram_tree, max_nodes: int = 16,
                         chunk: int = 0):
    """model.run_requests with drafted trees: the same output ids, in fewer
    steps where the guesses are good.  draft(tokens so far, most nodes) ->
    (node tokens, parents), node 0 the last token; ([], []) is no guess.  Returns
    (each request's output ids, model steps taken)."""
    for p in prompts:
        if len(p) + steps > dec.Lmax:
            raise ValueError("prompt empty or too long for the decoder's cache")
    dd = DraftDecoder(dec, max_nodes)
    dd.start(prompts, params, chunk=chunk)
    taken = 0
    while True:
        left = [steps - (len(seq) - n) for seq, n in zip(dd.requests, dd.prompt_len)]
        if all(x <= 0 for x in left):
            break
        trees = []
        for seq, more in zip(dd.requests, left):
            # no more nodes than the cache has slots for behind the request; without
            # a guess the step decides one token
            tree = draft(seq, min(max_nodes, dec.Lmax - len(seq) + 1)) if more > 0 else ([], [])
            trees.append(([seq[-1]], [-1]) if more > 0 and not tree[0] else tree)
        dd.step(trees)
        taken += 1
    return [seq[n: n + steps] for seq, n in zip(dd.requests, dd.prompt_len)], taken
