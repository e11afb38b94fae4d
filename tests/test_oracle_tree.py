"""The drafted-tree and log-probability oracles against closed forms and a
second way of saying the same thing."""
import numpy as np
import pytest
import torch

from helpers import synth
from oracle import attention as oattn, bf16 as obf, logprobs as olp, tree as otree


def test_paths_and_positions():
    parent = [-1, 0, 0, 1, 3, 2, -1, 6]
    assert otree.path_of(parent, 4) == [0, 1, 3, 4]
    assert otree.path_of(parent, 5) == [0, 2, 5]
    assert otree.path_of(parent, 7) == [6, 7]
    assert otree.positions(10, parent).tolist() == [10, 11, 11, 12, 13, 12, 10, 11]
    assert otree.valid(parent, 8) and not otree.valid([-1, 1], 2) and not otree.valid([-2], 1)
    with pytest.raises(ValueError):
        otree.path_of([-1, 2, 1], 2)


def test_a_chain_is_causal_prefill():
    n, ctx, hq, hkv, d = 5, 9, 4, 2, 64
    q = synth.bits(synth.normal_bf16((n, hq, d), 1.0, 1))
    k = synth.bits(synth.normal_bf16((ctx + n, hkv, d), 1.0, 2))
    v = synth.bits(synth.normal_bf16((ctx + n, hkv, d), 1.0, 3))
    chain = otree.attention(q, k, v, ctx, [-1, 0, 1, 2, 3])
    assert np.array_equal(chain, oattn.prefill(q, k, v, ctx))


def test_a_node_ignores_its_siblings():
    """Against a masked softmax written over all slots."""
    parent, ctx, hq, hkv, d = [-1, 0, 0, 2, 1, 2], 3, 2, 1, 64
    n = len(parent)
    q = synth.normal_bf16((n, hq, d), 1.0, 4)
    k, v = synth.normal_bf16((ctx + n, hkv, d), 1.0, 5), synth.normal_bf16((ctx + n, hkv, d), 1.0, 6)
    got = obf.to_f64(otree.attention(synth.bits(q), synth.bits(k), synth.bits(v), ctx, parent))
    sees = np.zeros((n, ctx + n), dtype=bool)
    sees[:, :ctx] = True
    for i in range(n):
        j = i
        while j >= 0:
            sees[i, ctx + j] = True
            j = parent[j]
    s = q.double().numpy() @ k.double().numpy()[:, 0].T / np.sqrt(d)
    s = np.where(sees[:, None], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    want = (p / p.sum(-1, keepdims=True)) @ v.double().numpy()[:, 0]
    assert np.abs(got - want).max() <= 2.0 ** -8 * np.abs(want).max()  # one bf16 rounding


def test_accept_walks_to_the_first_disagreement():
    parent = [-1, 0, 0, 1, 1, 4]
    tokens = [7, 5, 6, 5, 9, 2]
    assert otree.accept(parent, tokens, [5, 9, 0, 0, 2, 1]) == [0, 1, 4, 5]
    assert otree.accept(parent, tokens, [6, 9, 0, 0, 2, 1]) == [0, 2]
    assert otree.accept(parent, tokens, [8, 0, 0, 0, 0, 0]) == [0]
    assert otree.accept([-1, 0, 0], [1, 4, 4], [4, 0, 0]) == [0, 1]      # the lower of two equal children
    assert otree.accept([-1, -1], [1, 4], [4, 0]) == [0]                  # a second root follows nothing
    assert otree.accept([], [], []) == []


def test_logprobs_closed_forms():
    lp, h = olp.row(np.zeros(8))
    assert np.allclose(lp, -np.log(8)) and abs(h - np.log(8)) < 1e-14
    lp, h = olp.row(np.array([0.0, np.log(3.0)]))
    assert np.allclose(lp, [np.log(0.25), np.log(0.75)])
    assert abs(h - (np.log(4) - 0.75 * np.log(3))) < 1e-14
    lp, h = olp.row(np.array([1.0, np.nan, -np.inf, 1.0]))
    assert np.allclose(lp[[0, 3]], -np.log(2)) and np.all(lp[1:3] == -np.inf) and abs(h - np.log(2)) < 1e-14
    lp, h = olp.row(np.array([np.inf, 1.0, np.inf]))
    assert np.allclose(lp[[0, 2]], -np.log(2)) and lp[1] == -np.inf and abs(h - np.log(2)) < 1e-14
    lp, h = olp.row(np.full(3, -np.inf))
    assert np.all(lp == -np.inf) and h == 0
    x = torch.randn(1000, generator=synth.gen(1), dtype=torch.float64) * 4
    lp, h = olp.row(x.numpy())
    ref = torch.log_softmax(x, 0)
    assert np.allclose(lp, ref.numpy(), rtol=0, atol=1e-12)
    assert abs(h - float(-(ref.exp() * ref).sum())) < 1e-12
    assert olp.top(np.array([1.0, 3.0, 3.0, np.nan, 2.0]), 4).tolist() == [1, 2, 4, 0]
