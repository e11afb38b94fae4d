"""Calls on a named stream while the current one goes on: what the call allocates
and what it reads stays its own until it has run, and nothing that the current
stream still reads is written.  (The named stream is kept busy for some
milliseconds first, so that the call's kernels run after what follows here.)"""
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth
from test_gpu_tree import Case, shape_parents

pytestmark = gpu
BUSY = 20_000_000  # cycles, about ten milliseconds


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def tuple_of(out):
    return tuple(t for t in (out if isinstance(out, tuple) else (out,)) if t is not None)


def calls(kinv):
    """name -> (inputs, call(inputs, stream)); the inputs are all that the caller has."""
    c = Case(kinv, [3000, 300], [shape_parents("bushy", 40, 1), shape_parents("chain", 9)], 32, 8, 128, seed=400)
    t = c.tree
    tree = lambda x: kinv.Tree(*x, t.max_nodes, t.max_kv)
    small = Case(kinv, [200], [shape_parents("bushy", 4, 2)], 32, 8, 128, seed=401)
    ts = small.tree
    qkv = synth.normal_bf16((c.rows, 48 * 128), 1.0, 402, "cuda")
    tok, nxt = (synth.uniform_int(c.rows, 0, 2, s).to(torch.int32).cuda() for s in (403, 404))
    kv = torch.stack([c.k, c.v])[None].contiguous()
    x = torch.randn(64, 20000, generator=synth.gen(405, "cuda"), device="cuda")
    ids = synth.uniform_int(128, 0, 19999, 406).to(torch.int32).view(64, 2).cuda()

    def rope(i, s):
        q = torch.empty(c.rows, 32, 128, dtype=torch.bfloat16, device="cuda")
        kinv.rope_append_tree(i[0], q, i[1], i[2], tree(i[3:]), 32, 8, 128, 1e6, stream=s)
        return q, i[1], i[2]

    return {
        "attn_tree": ([c.q, c.k, c.v, *t.tensors], lambda i, s: kinv.attn_tree(*i[:3], tree(i[3:]), stream=s)),
        "attn_tree, one launch": ([small.q, small.k, small.v, *ts.tensors],
                                  lambda i, s: kinv.attn_tree(*i[:3], kinv.Tree(*i[3:], ts.max_nodes, ts.max_kv), stream=s)),
        "rope_append_tree": ([qkv, c.k, c.v, *t.tensors], rope),
        "tree_accept": ([tok, nxt, kv, *t.tensors], lambda i, s: (*kinv.tree_accept(tree(i[3:]), *i[:3], stream=s), i[2])),
        "logprobs": ([x, ids], lambda i, s: kinv.logprobs(*i, top_k=5, stream=s)),
    }


NAMES = ["attn_tree", "attn_tree, one launch", "rope_append_tree", "tree_accept", "logprobs"]


@pytest.mark.parametrize("name", NAMES)
def test_scratch_and_inputs_outlive_the_call(kinv, name):
    inputs, call = calls(kinv)[name]
    want = tuple_of(call([t.clone() for t in inputs], None))
    side = torch.cuda.Stream()
    for again in range(3):
        mine = [t.clone() for t in inputs]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        out = tuple_of(call(mine, side))
        sizes = [t.numel() * t.element_size() for t in mine] + [t.numel() * t.element_size() for t in want] + [1 << k for k in range(9, 27)]
        del mine
        new = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert_same_bits(a, b, f"{name}, {again}")
        del new, out
    assert kinv.last_device_status() == 0


@pytest.mark.parametrize("name", [n for n in NAMES if n != "rope_append_tree"])
def test_what_the_current_stream_still_reads_is_not_written(kinv, name):
    """Blocks of the outputs' and the scratch's sizes that the current stream has
    dropped but not read yet."""
    inputs, call = calls(kinv)[name]
    want = tuple_of(call(inputs if name != "tree_accept" else [t.clone() for t in inputs], None))
    sizes = [t.numel() * t.element_size() for t in want] * 2 + [1 << k for k in range(9, 27)]
    side = torch.cuda.Stream()
    mine = [t.clone() for t in inputs]
    dropped = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    read = [d.clone() for d in dropped]
    del dropped
    out = tuple_of(call(mine, side))
    torch.cuda.synchronize()
    for r in read:
        assert torch.all(r == 0x5A)
    for a, b in zip(out, want):
        assert_same_bits(a, b, name)
    # dropped here while the current stream has not read it: the side stream's next call leaves it alone
    ready = [[t.clone() for t in inputs] for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    read = [t.clone() for t in out]
    del out
    others = [tuple_of(call(i, side)) for i in ready]
    torch.cuda.synchronize()
    for a, b in zip(read, want):
        assert_same_bits(a, b, f"{name}, read late")
    del others
    assert kinv.last_device_status() == 0


def test_a_captured_call_on_a_stream_beside(kinv):
    """The same inside a graph: the call on a stream that joins the captured one."""
    inputs, call = calls(kinv)["attn_tree"]
    want = tuple_of(call(inputs, None))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        out = tuple_of(call(inputs, side))
        torch.cuda.current_stream().wait_stream(side)
        scratch = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        out[0].zero_()
        g.replay()
        assert_same_bits(out[0], want[0], "replayed")
    del scratch
    assert kinv.last_device_status() == 0


def test_decode_and_prefill_scratch_outlives_the_call(kinv):
    """The same for the attention calls whose scratch is allocated by default."""
    hq, hkv, d, lmax = 32, 8, 128, 4096
    k, v = (synth.normal_bf16((4, lmax, hkv, d), 1.0, s, "cuda") for s in (410, 411))
    q = synth.normal_bf16((4, hq, d), 1.0, 412, "cuda")
    n = torch.tensor([4096, 3000, 1, 700], dtype=torch.int32, device="cuda")
    start, lens, off = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (2000, 4, 0))
    side = torch.cuda.Stream()
    for call in (lambda s: kinv.attn_decode(q, k, v, n, stream=s),
                 lambda s: kinv.attn_prefill(q, k, v, start, lens, off, 4, 2004, stream=s)):
        want = call(None)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        out = call(side)
        new = [torch.full((1 << b,), 0xFF, dtype=torch.uint8, device="cuda") for b in range(9, 27) for _ in range(2)]
        torch.cuda.synchronize()
        assert_same_bits(out, want)
        del new
    assert kinv.last_device_status() == 0
