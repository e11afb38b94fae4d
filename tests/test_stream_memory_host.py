"""Memory of a call on a named stream (no GPU: tensors, streams and the library
are stand-ins that record what is asked of them).  What a call allocates has to
come from that stream's memory -- the current stream's allocator may hand out a
freed block again before the named stream has run -- and what it reads has to
be held for that stream."""
import types

import pytest
import torch

from invariant_deterministic_gb300 import kinv

BF, I32, F32, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
SIDE = types.SimpleNamespace(cuda_stream=7)
MAIN = types.SimpleNamespace(cuda_stream=3)


class Tensor:
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype, made_on=None):
        self.shape, self.dtype, self.made_on, self.held = tuple(shape), dtype, made_on, []

    def stride(self, i=None):
        s, at = [], 1
        for n in reversed(self.shape):
            s.insert(0, at)
            at *= n
        return tuple(s) if i is None else s[i]

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def element_size(self):
        return {BF: 2, U8: 1}.get(self.dtype, 4)

    def data_ptr(self):
        return 4096

    def record_stream(self, s):
        self.held.append(s)


@pytest.fixture
def world(monkeypatch):
    made, now = [], [MAIN]

    def make(*shape, dtype=None, device=None, **kw):
        shape = shape[0] if len(shape) and isinstance(shape[0], (tuple, list)) else shape
        made.append(Tensor(shape, dtype, now[0]))
        return made[-1]

    class On:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.was, now[0] = now[0], self.s

        def __exit__(self, *exc):
            now[0] = self.was

    class Torch:
        empty = staticmethod(make)
        cuda = types.SimpleNamespace(stream=On, current_stream=lambda device=None: now[0])

        @staticmethod
        def empty_like(t):
            return make(t.shape, dtype=t.dtype)

        def __getattr__(self, name):
            return getattr(torch, name)

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: 4096) if name.endswith("_workspace") else (lambda *a: calls.append((name, a)) or 0)

    calls = []
    monkeypatch.setattr(kinv, "torch", Torch())
    monkeypatch.setattr(kinv, "_raw_stream", None)
    monkeypatch.setattr(kinv, "lib", lambda: Lib())
    return types.SimpleNamespace(made=made, calls=calls)


def tree():
    return kinv.Tree(Tensor((2,), I32), Tensor((2,), I32), Tensor((2,), I32), Tensor((10,), I32), 8, 512)


def drafted_calls():
    """name -> (call with a stream, tensors it reads or writes of the caller's)"""
    t = tree()
    k, v = Tensor((2, 512, 2, 64), BF), Tensor((2, 512, 2, 64), BF)
    q, qkv, gains = Tensor((10, 4, 64), BF), Tensor((10, 512), BF), [Tensor((64,), BF), Tensor((64,), BF)]
    tok, nxt, kv = Tensor((10,), I32), Tensor((10,), I32), Tensor((3, 2, 2, 512, 2, 64), BF)
    x, ids = Tensor((3, 100), F32), Tensor((3, 2), I32)
    ws = Tensor((8192,), U8)
    return {
        "attn_tree": (lambda s: kinv.attn_tree(q, k, v, t, stream=s), [q, k, v, *t.tensors]),
        "attn_tree, scratch given": (lambda s: kinv.attn_tree(q, k, v, t, workspace=ws, stream=s), [q, k, v, ws, *t.tensors]),
        "rope_append_tree": (lambda s: kinv.rope_append_tree(qkv, q, k, v, t, 4, 2, 64, 1e4, *gains, stream=s),
                             [qkv, q, k, v, *gains, *t.tensors]),
        "tree_accept": (lambda s: kinv.tree_accept(t, tok, nxt, kv, stream=s), [tok, nxt, kv, *t.tensors]),
        "logprobs": (lambda s: kinv.logprobs(x, ids, top_k=5, stream=s), [x, ids]),
    }


@pytest.mark.parametrize("name", list(drafted_calls()))
def test_drafted_and_scoring_calls_on_a_named_stream(world, name):
    call, inputs = drafted_calls()[name]
    out = call(SIDE)
    (_, args), = world.calls
    assert args[-1] == SIDE.cuda_stream
    assert all(t.made_on is SIDE for t in world.made), "memory of another stream than the call's"
    for t in inputs:
        assert SIDE in t.held, "an input that may be dropped under the running kernel"
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and t.made_on is not None:
            assert MAIN in t.held, "an output that the current stream reads and may drop"


@pytest.mark.parametrize("name", list(drafted_calls()))
@pytest.mark.parametrize("stream", [None, MAIN])
def test_on_the_current_stream_nothing_is_held(world, name, stream):
    call, inputs = drafted_calls()[name]
    call(stream)
    assert world.calls[0][1][-1] == MAIN.cuda_stream
    assert all(t.made_on is MAIN and not t.held for t in world.made) and not any(t.held for t in inputs)


def other_calls():
    a, w, row, q = Tensor((4, 256), BF), Tensor((256, 256), BF), Tensor((256,), BF), Tensor((3, 4, 64), BF)
    k, v, n = Tensor((3, 512, 2, 64), BF), Tensor((3, 512, 2, 64), BF), Tensor((3,), I32)
    x, h = Tensor((3, 100), F32), Tensor((3, 64), I32)
    return {
        "gemm": lambda s: kinv.gemm(a, w, stream=s),
        "gemm_swiglu": lambda s: kinv.gemm_swiglu(a, w, stream=s),
        "rmsnorm": lambda s: kinv.rmsnorm(a, row, stream=s),
        "attn_decode": lambda s: kinv.attn_decode(q, k, v, n, stream=s),
        "attn_prefill": lambda s: kinv.attn_prefill(q, k, v, n, n, n, 3, 512, stream=s),
        "sample": lambda s: kinv.sample(x, row, h, n, n, stream=s),
        "embed": lambda s: kinv.embed(w, n, stream=s),
        "add": lambda s: kinv.add(a, a, stream=s),
        "scale_columns": lambda s: kinv.scale_columns(w, row, stream=s),
        "swiglu": lambda s: kinv.swiglu(a, stream=s),
    }


@pytest.mark.parametrize("name", list(other_calls()))
def test_other_calls_allocate_on_their_stream(world, name):
    out = other_calls()[name](SIDE)
    assert world.calls[0][1][-1] == SIDE.cuda_stream
    assert world.made and all(t.made_on is SIDE for t in world.made)
    assert out.made_on is SIDE and MAIN in out.held
    world.made.clear()
    out = other_calls()[name](None)
    assert world.calls[1][1][-1] == MAIN.cuda_stream and all(t.made_on is MAIN and not t.held for t in world.made)


@pytest.mark.parametrize("given", [(), ("path",), ("out_tokens",), ("n_accepted",), ("n_accepted", "path", "out_tokens")])
def test_allocated_results_are_defined_for_a_sequence_left_out(world, given):
    """The kernel marks the outputs that were allocated, and leaves those that were given."""
    tok = Tensor((10,), I32)
    mine = {name: Tensor((16,), I32) for name in given}
    out = dict(zip(("n_accepted", "path", "out_tokens"), kinv.tree_accept(tree(), tok, tok, **mine)))
    (name, args), = world.calls
    assert name == "kinv_tree_accept_marked"
    assert args[-2] == sum(bit for bit, x in ((1, "n_accepted"), (2, "path"), (4, "out_tokens")) if x not in given)
    for x in given:
        assert out[x] is mine[x]
