"""The drafter's trees and the checks of drafted steps (no GPU)."""
import pytest

from invariant_deterministic_gb300 import draft


def _paths(nodes, parents):
    out = []
    for i in range(len(nodes)):
        p, j = [], i
        while j >= 0:
            p.insert(0, nodes[j])
            j = parents[j]
        out.append(p)
    return out


def test_ngram_tree_follows_earlier_occurrences():
    #        0  1  2  3  4  5  6  7  8
    tokens = [1, 2, 3, 9, 1, 2, 4, 1, 2]
    nodes, parents = draft.ngram_tree(tokens, 64, n=2, depth=3)
    paths = _paths(nodes, parents)
    assert nodes[0] == 2 and parents[0] == -1
    assert [2, 4, 1, 2] in paths and [2, 3, 9, 1] in paths     # after (1, 2): the latest first
    assert all(0 <= p < i for i, p in enumerate(parents) if i)
    assert len({tuple(p) for p in paths}) == len(paths)         # no two nodes say the same


@pytest.mark.parametrize("most", [1, 2, 3, 5])
def test_ngram_tree_keeps_its_size(most):
    nodes, parents = draft.ngram_tree([5, 6] * 10, most)
    assert 1 <= len(nodes) <= most and len(nodes) == len(parents)


def test_ngram_tree_without_an_occurrence():
    assert draft.ngram_tree([7], 8) == ([7], [-1])
    assert draft.ngram_tree([1, 2, 3], 8) == ([3], [-1])


class _Dec:
    B, Lmax, hist_ld, max_rows = 2, 10, 4, 8

    class s:
        vocab = 100


def _dd(requests):
    d = draft.DraftDecoder.__new__(draft.DraftDecoder)
    d.dec, d.max_nodes, d.requests, d.prompt_len = _Dec, 4, requests, [2] * len(requests)
    return d


def test_step_inputs():
    d = _dd([[1, 2, 3], [8, 9]])
    token, parent, owner, step, n, hist, hist_len = d._inputs([([3, 4, 5, 6], [-1, 0, 0, 2]), ([], [])])
    assert token == [3, 4, 5, 6] and parent == [-1, 0, 0, 2] and owner == [0] * 4 and n == [4, 0]
    assert step == [1, 2, 2, 3]                                  # one token decided, then the path's
    assert hist[0] == [1, 2, 3, 0] and hist_len[0] == 3
    assert hist[1] == [1, 2, 3, 4] and hist[3] == [2, 3, 5, 6] and hist_len[3] == 4


@pytest.mark.parametrize("tree", [([4], [-1]), ([3], [0]), ([3, 4], [-1]), ([3] * 5, [-1, 0, 1, 2, 3]),
                                  ([3, 4], [-1, 1]), ([3, 4], [-1, -1]), ([3, -1], [-1, 0]), ([3, 100], [-1, 0])])
def test_step_refuses_broken_trees(tree):
    with pytest.raises(ValueError):
        _dd([[1, 2, 3]])._inputs([tree])


def test_step_needs_a_tree_per_request():
    d = _dd([[1, 2, 3], [8, 9]])
    for trees in ([], [([3], [-1])], [([3], [-1]), ([9], [-1]), ([], [])]):
        with pytest.raises(ValueError):
            d.step(trees)


def test_step_refuses_a_tree_past_the_cache():
    with pytest.raises(ValueError):
        _dd([list(range(9))])._inputs([([8, 1, 2], [-1, 0, 1])])


def test_decoder_limits():
    class D:
        B, max_rows = 4, 63
    with pytest.raises(ValueError):
        draft.DraftDecoder(D, 16)
    with pytest.raises(ValueError):
        draft.DraftDecoder(D, 65)


class _Steps:
    """Stands in for DraftDecoder: a step decides the next tokens of a fixed answer,
    as many as the tree's chain from node 0 gets right, and one more."""

    def __init__(self, dec, max_nodes):
        self.most, self.trees = max_nodes, []

    def start(self, prompts, params, chunk=0):
        self.requests = [list(p) for p in prompts]
        self.prompt_len = [len(p) for p in prompts]

    def step(self, trees):
        for seq, (nodes, parents) in zip(self.requests, trees):
            if nodes:
                assert nodes[0] == seq[-1] and parents[0] == -1 and len(nodes) <= self.most
                last, right = seq[-1], 0
                while right + 1 < len(nodes) and nodes[right + 1] == last + right + 1:
                    right += 1
                seq.extend(range(last + 1, last + right + 2))
        self.trees.append(trees)


def _drafted(monkeypatch, prompts, steps, guess):
    monkeypatch.setattr(draft, "DraftDecoder", _Steps)
    return draft.run_requests_drafted(_Dec, prompts, None, steps, draft=guess, max_nodes=4)


def test_a_drafter_with_no_guess_leaves_the_answer_whole(monkeypatch):
    prompts, want = [[1, 2], [7]], [[3, 4, 5, 6], [8, 9, 10, 11]]
    assert _drafted(monkeypatch, prompts, 4, lambda t, n: ([], [])) == (want, 4)
    # no guess for one request, in some of its steps, or in all but the first
    assert _drafted(monkeypatch, prompts, 4, lambda t, n: ([], []) if t[0] == 7 else ([t[-1]], [-1])) == (want, 4)
    once = lambda t, n: ([t[-1], t[-1] + 1], [-1, 0]) if len(t) < 3 else ([], [])
    assert _drafted(monkeypatch, prompts, 4, once)[0] == want
    assert _drafted(monkeypatch, prompts, 0, lambda t, n: ([], [])) == ([[], []], 0)
