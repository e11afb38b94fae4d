"""Drafted trees through the whole model: the tokens, the logits' bits and the
cache of decoding one token at a time; scores of a prompt."""
import numpy as np
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth
from oracle import logprobs as olp

pytestmark = gpu


@pytest.fixture(scope="module")
def M():
    ensure_lib()
    from invariant_deterministic_gb300 import draft, model
    model.draft = draft
    return model


def _shape(M, name):
    if name == "tiny":
        return M.TINY
    return M.ModelShape(**{**M.QWEN3_8B.__dict__, "n_layers": 2, "vocab": 2048})


def _params(M, n):
    # each request its own settings; low temperatures repeat themselves, so lookups hit
    kinds = [dict(temperature=0.0, repeat_penalty=1.0), dict(temperature=0.8), dict(temperature=0.3, repeat_penalty=1.0),
             dict(temperature=1.0, presence_penalty=0.5, frequency_penalty=0.2, repeat_last_n=16)]
    return [M.kinv.SamplingParams(seed=1000 + i, **kinds[i % 4]) for i in range(n)]


def _prompts(shape, n):
    return [synth.uniform_int(5 + 37 * i, 0, shape.vocab - 1, 50 + i).tolist() for i in range(n)]


def _guesser(answers, prompts, wrong_from):
    """A drafter that knows the answers: right up to a point of each tree, with
    wrong siblings; node 0 is the last token."""
    def draft(tokens, max_nodes):
        i = next(k for k, p in enumerate(prompts) if tokens[: len(p)] == p)
        done = len(tokens) - len(prompts[i])
        nodes, parents, at = [tokens[-1]], [-1], 0
        for k, t in enumerate(answers[i][done: done + 6]):
            if len(nodes) + 2 > max_nodes:
                break
            nodes.append((t + 1) % 512), parents.append(at)          # a wrong sibling first
            nodes.append(t if k < wrong_from else (t + 2) % 512), parents.append(at)
            at = len(nodes) - 1
        return nodes, parents
    return draft


@pytest.mark.parametrize("name", ["tiny", "8b wide"])
def test_drafted_decoding_gives_the_tokens_and_the_cache_of_decoding(M, name):
    shape = _shape(M, name)
    w = M.random_weights(shape, device="cuda")
    prompts, steps, lmax, nodes = _prompts(shape, 4), 40, 400, 16
    params = _params(M, 4)
    dec = M.Decoder(shape, w, max_batch=4, max_len=lmax, max_chunk=64)
    want = M.run_requests(dec, prompts, params, steps)
    plain = dec.kv.clone()
    for draft, most in ((M.draft.ngram_tree, steps), (_guesser(want, prompts, 99), steps - 1),
                        (_guesser(want, prompts, 2), steps - 1), (lambda t, n: ([t[-1]], [-1]), steps)):
        d2 = M.Decoder(shape, w, max_batch=4, max_len=lmax, max_chunk=64)
        got, taken = M.draft.run_requests_drafted(d2, prompts, params, steps, draft=draft, max_nodes=nodes)
        assert got == want
        assert taken <= most  # right guesses are taken
        # the cache of all but the last token (which neither run has put there)
        for b, p in enumerate(prompts):
            n = len(p) + steps - 1
            assert_same_bits(d2.kv[:, :, b, :n], plain[:, :, b, :n], f"cache of request {b}")
        assert M.kinv.last_device_status() == 0


def test_a_nodes_logits_have_the_bits_of_decode(M):
    shape = _shape(M, "8b wide")
    w = M.random_weights(shape, device="cuda")
    dec = M.Decoder(shape, w, max_batch=2, max_len=700, max_chunk=64)
    prompts = [synth.uniform_int(n, 0, shape.vocab - 1, n).tolist() for n in (300, 511)]
    dd = M.draft.DraftDecoder(dec, 16)
    dd.start(prompts, _params(M, 2))
    trees = [([prompts[0][-1], 5, 9, 7, 5], [-1, 0, 0, 2, 3]), ([prompts[1][-1], 3], [-1, 0])]
    dd.step(trees)
    logits = dd.logits[:7].clone()
    row = 0
    for b, (nodes, parents) in enumerate(trees):
        for i in range(len(nodes)):
            path, j = [], i
            while j > 0:
                path.insert(0, nodes[j])
                j = parents[j]
            d2 = M.Decoder(shape, w, max_batch=1, max_len=700, max_chunk=512)
            seq = prompts[b] + path
            d2.prefill(0, torch.tensor(seq[:-1], dtype=torch.int32, device="cuda"))
            d2.set_positions([len(seq) - 1])
            d2.tokens[0] = seq[-1]
            d2.decode_step(1, sample=False)
            assert_same_bits(logits[row], d2.logits[0], f"request {b} node {i}")
            row += 1


def test_score_of_a_prompt(M):
    shape = _shape(M, "tiny")
    w = M.random_weights(shape, device="cuda")
    tokens = synth.uniform_int(130, 0, shape.vocab - 1, 3).cuda()
    dec = M.Decoder(shape, w, max_batch=3, max_len=200, max_chunk=64)
    lp, ent, ids, top = dec.score(1, tokens, top_k=4)
    assert lp.shape == (129,) and ids.shape == (129, 4)
    for chunk in (7, 64):
        for a, b in zip(dec.score(0, tokens, top_k=4, chunk=chunk), (lp, ent, ids, top)):
            assert_same_bits(a, b, f"chunk {chunk}")
    # against the logits of decode steps over the same tokens
    d2 = M.Decoder(shape, w, max_batch=1, max_len=200)
    for i in range(0, 129, 16):
        if i:
            d2.prefill(0, tokens[:i], chunk=1)
        d2.set_positions([i])
        d2.tokens[0] = tokens[i]
        d2.decode_step(1, sample=False)
        full, h = olp.row(d2.logits[0].cpu().numpy())
        # tolerance of kinv_logprobs over 512 ids, derived in test_gpu_logprobs.py
        assert abs(lp[i].item() - full[int(tokens[i + 1])]) <= 8.2e-6 + 2.0 ** -22 * abs(lp[i].item())
        assert abs(ent[i].item() - h) <= 2.1e-4
        assert ids[i].tolist() == olp.top(d2.logits[0].cpu().numpy(), 4).tolist()
    for seq, n, chunk in ((0, 1, 0), (3, 9, 0), (-1, 9, 0), (0, 9, -1)):
        with pytest.raises(ValueError):
            dec.score(seq, tokens[:n], chunk=chunk)
    # the whole cache, and one more token than it can score
    long = synth.uniform_int(202, 0, shape.vocab - 1, 4).cuda()
    assert dec.score(2, long[:201])[0].shape == (200,)
    with pytest.raises(ValueError):
        dec.score(2, long)
    # more rows than the logits hold at a time
    M.SCORE_ROWS, rows = 20, M.SCORE_ROWS
    try:
        for a, b in zip(dec.score(1, tokens, top_k=4), (lp, ent, ids, top)):
            assert_same_bits(a, b, "twenty rows at a time")
    finally:
        M.SCORE_ROWS = rows
