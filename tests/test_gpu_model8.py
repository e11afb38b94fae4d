"""The decoder over 8-bit caches and windowed attention: what it attends to is the
definition's, a request's bits do not depend on batch, slot, chunking or on whether
a row is prefilled or decoded, and prefixes, scoring, receipts and graphs work as
with a bf16 cache."""
import json

import numpy as np
import pytest
import torch

from helpers import assert_close, assert_same_bits, ensure_lib, f64, gpu, synth
from invariant_deterministic_gb300 import receipt
from oracle import cache8 as o8, window as owin

pytestmark = gpu

I32 = dict(dtype=torch.int32, device="cuda")
# cache, window, sinks: a window that ends inside a split, one over several splits
KINDS = [("e4m3", 0, 0), ("int8", 0, 0), ("bf16", 24, 2), ("e4m3", 300, 4), ("int8", 40, 1)]


@pytest.fixture(scope="module")
def M():
    ensure_lib()
    from invariant_deterministic_gb300 import model
    return model


def shape_of(M, window, sinks, layers=2):
    return M.ModelShape(d_model=256, n_q=4, n_kv=2, head_dim=64, ffn=512, vocab=512, n_layers=layers, qk_norm=True, window=window, sinks=sinks)


@pytest.fixture(scope="module")
def weights(M):
    return M.random_weights(shape_of(M, 0, 0))


def decoder(M, weights, kind, batch=4, length=640, chunk=256):
    cache, window, sinks = kind
    return M.Decoder(shape_of(M, window, sinks), weights, max_batch=batch, max_len=length, max_chunk=chunk, cache=cache)


def cache_tensors(dec):
    return [dec.kv] if dec.cache == "bf16" else [dec.kv.view(torch.uint8), dec.kv_exp]


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_a_step_attends_to_what_the_cache_holds(M, weights, kind):
    """One decode step's attention against the fp64 definition over the held values."""
    cache, window, sinks = kind
    dec = decoder(M, weights, kind)
    lens = [1, 23, 300, 555]
    for b, n in enumerate(lens):
        dec.prefill(b, synth.uniform_int(n, 0, 511, 30 + b).cuda(), chunk=200)
    dec.set_positions(lens)
    dec.tokens[:4] = torch.tensor([5, 6, 7, 8], **I32)
    dec.decode_step(4, sample=False)
    assert M.kinv.last_device_status() == 0
    li = 1   # q and attn hold the last layer's
    for b, n in enumerate(lens):
        if cache == "bf16":
            k, v = f64(dec.kv[li, 0, b]), f64(dec.kv[li, 1, b])
        else:
            k, v = (o8.values(dec.kv[li, i, b].view(torch.uint8).cpu().numpy(), dec.kv_exp[li, i, b].T.cpu().numpy(), cache) for i in (0, 1))
        ref = owin.row(f64(dec.q[b]), k, v, n, window, sinks)
        assert_close(f64(dec.attn[b]), ref, f"sequence {b}")


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_bits_do_not_depend_on_chunks_slots_or_the_kind_of_step(M, weights, kind):
    n = 560
    prompt = synth.uniform_int(n, 0, 511, 40).cuda()
    dec = decoder(M, weights, kind)
    whole = dec.prefill(0, prompt, chunk=256)
    tensors = [t[:, :, 0].clone() for t in cache_tensors(dec)]
    for slot, chunk in ((1, 64), (2, 7)):
        assert_same_bits(dec.prefill(slot, prompt, chunk=chunk), whole, f"chunks of {chunk}")
        for t, ref in zip(cache_tensors(dec), tensors):
            assert_same_bits(t[:, :, slot], ref, f"cache after chunks of {chunk}")
    # the last token as a decode step, beside other requests
    dec.prefill(3, prompt[: n - 1])
    for b, m in ((0, 100), (1, 3), (2, 333)):
        dec.prefill(b, synth.uniform_int(m, 0, 511, 41 + b).cuda())
    dec.set_positions([100, 3, 333, n - 1])
    dec.tokens[:4] = torch.tensor([1, 2, 3, int(prompt[-1])], **I32)
    dec.decode_step(4, sample=False)
    assert_same_bits(dec.x[3], whole, "decode step")
    for t, ref in zip(cache_tensors(dec), tensors):
        assert_same_bits(t[:, :, 3], ref, "cache after the decode step")
    assert M.kinv.last_device_status() == 0


@pytest.mark.parametrize("kind", KINDS[:1] + KINDS[2:4], ids=str)
def test_requests_alone_together_and_captured(M, weights, kind):
    lens, steps = [3, 200, 31, 290], 12
    prompts = [synth.uniform_int(m, 0, 511, 50 + i).tolist() for i, m in enumerate(lens)]
    params = [M.kinv.SamplingParams(seed=70 + i) for i in range(4)]
    dec = decoder(M, weights, kind)
    together = M.run_requests(dec, prompts, params, steps, chunk=100)
    for i in (1, 2):
        assert M.run_requests(decoder(M, weights, kind, batch=1), [prompts[i]], [params[i]], steps)[0] == together[i]
    # the same steps replayed from a graph
    dec = decoder(M, weights, kind)
    for i, p in enumerate(prompts):
        dec.prefill(i, torch.tensor(p[:-1], **I32))
    dec.set_sampling(params)

    def state():
        dec.set_history(prompts)
        dec.set_positions([m - 1 for m in lens])
        dec.step[:4] = 0
        dec.tokens[:4] = torch.tensor([p[-1] for p in prompts], **I32)
    state()
    dec.decode_step(4)
    torch.cuda.synchronize()
    state()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.decode_step(4)
    state()
    got = []
    for _ in range(steps):
        g.replay()
        got.append(dec.tokens[:4].tolist())
    assert [list(x) for x in zip(*got)] == together
    assert M.kinv.last_device_status() == 0


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_prefixes_are_reused_read_and_loaded(M, weights, kind):
    prompt = synth.uniform_int(300, 0, 511, 60).cuda()
    dec = decoder(M, weights, kind)
    pc = M.PrefixCache(dec)
    whole = dec.prefill(0, prompt)
    pc.insert(prompt[:260].tolist(), 0)
    used, got = pc.prefill(2, prompt)
    assert used == 260
    assert_same_bits(got, whole, "reused prefix")
    k, v = dec.read_prefix(0, 260)
    other = decoder(M, weights, kind)
    other.load_prefix(1, k, v)
    assert_same_bits(other.prefill(1, prompt[260:], p0=260), whole, "loaded prefix")
    # from the host, the values in another order of memory than the keys
    third = decoder(M, weights, kind)
    third.load_prefix(1, k.cpu(), v.transpose(1, 2).contiguous().transpose(1, 2))
    for a, b in zip(third.read_prefix(1, 260), (k, v)):
        assert_same_bits(a, b, "loaded from elsewhere")
    for bad in (dict(seq=4, n=3), dict(seq=0, n=641), dict(seq=0, n=-1)):
        with pytest.raises(ValueError):
            dec.read_prefix(**bad)
    with pytest.raises(ValueError):
        dec.load_prefix(0, k[:1], v[:1])


def test_scores_and_receipts(M, weights):
    tokens = synth.uniform_int(150, 0, 511, 61).cuda()
    dec = decoder(M, weights, ("int8", 40, 1))
    lp, ent, _, _ = dec.score(1, tokens, chunk=64)
    lp2, ent2, _, _ = dec.score(2, tokens, chunk=17)
    assert_same_bits(lp, lp2, "score")
    assert torch.isfinite(lp).all() and torch.isfinite(ent).all()
    kinv = M.kinv
    for kind in (("e4m3", 0, 0), ("bf16", 24, 2)):
        shape = shape_of(M, kind[1], kind[2])
        prompt = synth.uniform_int(90, 0, 511, 62).tolist()
        p = kinv.SamplingParams(seed=9)
        outs = M.run_requests(decoder(M, M.random_weights(shape, seed=0), kind), [prompt[:20], prompt], [p, p], 10)
        r = receipt.make_receipt(build_id=kinv.build_id(), device_class=kinv.device_class(), settings=receipt.settings_of(shape, kind[0]),
                                 prompt_ids=prompt, sampling=p.__dict__, output_ids=outs[1], model=receipt.model_identity(shape, 0))
        r = json.loads(receipt.dumps(r))
        assert receipt.verify(r).startswith("identical, 10 of 10")
        r["device"]["settings"]["cache"] = "e5m2"
        assert receipt.verify(r).startswith("refused")


def test_rounding_the_cache_moves_the_logits_little(M, weights):
    """The 8-bit caches against the bf16 one: a code is off by at most half a step
    (2^-4 of the value for e4m3, 2^-7 of the vector's largest for int8), so every
    value that attention mixes is, and the logits stay near; int8 nearer, as its
    vectors here have no loud channels."""
    prompt = synth.uniform_int(200, 0, 511, 63).cuda()
    out = {}
    for kind in (("bf16", 0, 0), ("e4m3", 0, 0), ("int8", 0, 0)):
        dec = decoder(M, weights, kind)
        dec.prefill(0, prompt[:-1])
        dec.set_positions([199])
        dec.tokens[0] = prompt[-1]
        dec.decode_step(1, sample=False)
        out[kind[0]] = f64(dec.logits[0])
    rel = {c: np.linalg.norm(out[c] - out["bf16"]) / np.linalg.norm(out["bf16"]) for c in ("e4m3", "int8")}
    assert 0 < rel["int8"] < rel["e4m3"] < 2.0 ** -4, rel


def test_what_has_no_such_form_is_refused(M, weights):
    from invariant_deterministic_gb300 import draft
    with pytest.raises(ValueError):
        decoder(M, weights, ("e5m2", 0, 0))
    with pytest.raises(ValueError):
        decoder(M, weights, ("bf16", -1, 0))
    for kind in (("e4m3", 0, 0), ("bf16", 24, 0)):
        with pytest.raises(ValueError):
            draft.DraftDecoder(decoder(M, weights, kind), max_nodes=4)
        with pytest.raises(ValueError):
            decoder(M, weights, kind).tree_layers(None, 1, None)
