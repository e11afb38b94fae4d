"""Drafted decoding in caches of thousands of slots: the tensor-core kernel for the
context, reached through the model, beside requests that are still short."""
import pytest
import torch

from helpers import assert_same_bits, gpu, synth
from test_gpu_draft import M, _guesser, _params, _shape  # noqa: F401

pytestmark = gpu


@pytest.mark.parametrize("lens,lmax,nodes", [((2500, 700, 5, 1200), 2600, 16), ((300,), 32768, 8), ((9000, 40), 9100, 64)])
def test_drafted_decoding_in_a_large_cache(M, lens, lmax, nodes):  # noqa: F811
    shape = _shape(M, "8b wide")
    w = M.random_weights(shape, device="cuda")
    prompts, steps = [synth.uniform_int(n, 0, shape.vocab - 1, 600 + n).tolist() for n in lens], 24
    params = _params(M, len(lens))
    dec = M.Decoder(shape, w, max_batch=len(lens), max_len=lmax, max_chunk=256)
    want = M.run_requests(dec, prompts, params, steps)
    plain = dec.kv.clone()
    for draft in (_guesser(want, prompts, 99), _guesser(want, prompts, 1), M.draft.ngram_tree):
        d2 = M.Decoder(shape, w, max_batch=len(lens), max_len=lmax, max_chunk=256)
        got, taken = M.draft.run_requests_drafted(d2, prompts, params, steps, draft=draft, max_nodes=nodes)
        assert got == want and taken <= steps
        for b, n in enumerate(lens):
            assert_same_bits(d2.kv[:, :, b, : n + steps - 1], plain[:, :, b, : n + steps - 1], f"cache of request {b}")
        del d2
    assert M.kinv.last_device_status() == 0
