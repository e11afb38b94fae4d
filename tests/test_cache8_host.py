"""The 8-bit cache's and the windowed calls' Python side (no GPU: the library and
the streams are stand-ins that record what is asked of them): the stream that a
call's memory belongs to, and what is refused before the library is called."""
import types

import pytest
import torch

from invariant_deterministic_gb300 import kinv
from test_stream_memory_host import BF, F32, I32, MAIN, SIDE, U8, Tensor, world  # noqa: F401

E4 = torch.float8_e4m3fn


class Here(Tensor):
    """A stand-in on device 0, with the strides that it is given."""

    def __init__(self, shape, dtype, strides=None, device=0):
        super().__init__(shape, dtype)
        self.strides, self.index, self.device = strides, device, f"cuda:{device}"

    def get_device(self):
        return self.index

    def stride(self, i=None):
        if self.strides is None:
            return super().stride(i)
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return self.strides is None

    def element_size(self):
        return 1 if self.dtype in (E4, torch.int8) else super().element_size()


@pytest.fixture
def here(world, monkeypatch):  # noqa: F811
    monkeypatch.setattr(kinv, "_get_device", lambda: 0)
    monkeypatch.setattr(Tensor, "get_device", lambda self: 0, raising=False)
    return world


def args():
    """The tensors of a call, by name."""
    v = Here((3,), I32)
    a = dict(q=Here((3, 4, 64), BF), k=Here((3, 512, 2, 64), BF), v=Here((3, 512, 2, 64), BF), n=v, start=Here((3,), I32),
             off=Here((3,), I32), ws=Here((1 << 20,), U8), out=Here((3, 4, 64), BF), qkv=Here((3, 512), BF), gain=Here((64,), BF),
             ck=Here((3, 512, 2, 64), E4), cv=Here((3, 512, 2, 64), E4), ke=Here((3, 2, 512), torch.int8), ve=Here((3, 2, 512), torch.int8))
    return a


def cache(a):
    return kinv.Cache8(a["ck"], a["cv"], a["ke"], a["ve"])


CALLS = {
    "attn_decode": (lambda a, s, **kw: kinv.attn_decode(a["q"], a["k"], a["v"], a["n"], window=9, stream=s, **kw), "q k v n"),
    "attn_prefill": (lambda a, s, **kw: kinv.attn_prefill(a["q"], a["k"], a["v"], a["start"], a["n"], a["off"], 3, 512, window=9, stream=s, **kw),
                     "q k v start n off"),
    "attn_decode8": (lambda a, s, **kw: kinv.attn_decode8(a["q"], cache(a), a["n"], stream=s, **kw), "q ck cv ke ve n"),
    "attn_prefill8": (lambda a, s, **kw: kinv.attn_prefill8(a["q"], cache(a), a["start"], a["n"], a["off"], 3, 512, stream=s, **kw),
                      "q ck cv ke ve start n off"),
    "rope_append8": (lambda a, s: kinv.rope_append8(a["qkv"], a["out"], cache(a), a["n"], a["start"], 4, 2, 64, 1e4, a["gain"], a["gain"], stream=s),
                     "qkv out ck cv ke ve n start gain"),
    "cache8_write": (lambda a, s: kinv.cache8_write(cache(a), a["k"], a["v"], a["start"], a["n"], stream=s), "ck cv ke ve k v start n"),
    "cache8_read": (lambda a, s: kinv.cache8_read(cache(a), a["start"], a["n"], 512, stream=s), "ck cv ke ve start n"),
    "cache8_read into tensors": (lambda a, s: kinv.cache8_read(cache(a), a["start"], a["n"], k=a["k"], v=a["v"], stream=s),
                                 "ck cv ke ve k v start n"),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_on_a_named_stream(here, name):
    call, used = CALLS[name]
    a = args()
    out = call(a, SIDE)
    assert here.calls[0][1][-1] == SIDE.cuda_stream
    assert all(t.made_on is SIDE for t in here.made), "memory of another stream than the call's"
    for x in used.split():
        assert SIDE in a[x].held, f"{x} may be dropped under the running kernel"
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and t.made_on is not None:
            assert MAIN in t.held, "an output that the current stream reads and may drop"


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream", [None, MAIN])
def test_on_the_current_stream_nothing_is_held(here, name, stream):
    call, _ = CALLS[name]
    a = args()
    call(a, stream)
    assert here.calls[0][1][-1] == MAIN.cuda_stream
    assert all(t.made_on is MAIN and not t.held for t in here.made) and not any(t.held for t in a.values())


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_another_device_are_refused(here, name):
    call, used = CALLS[name]
    for x in used.split():
        a = args()
        a[x].index, a[x].device = 1, "cuda:1"
        with pytest.raises(ValueError):
            call(a, None)
        a[x].index, a[x].device = -1, "cpu"
        with pytest.raises(ValueError):
            call(a, None)
    a = args()
    for x in used.split():          # all on one device, which is not the current one
        a[x].index, a[x].device = 1, "cuda:1"
    with pytest.raises(ValueError):
        call(a, None)
    assert not here.calls


WRONG = {
    "q": [((3, 4), BF, None), ((3, 4, 64), F32, None), ((3, 4, 64), BF, (512, 64, 1)), ((3, 4, 128), BF, None)],
    "k": [((3, 512, 2), BF, None), ((3, 512, 2, 64), F32, None), ((3, 512, 2, 64), BF, (1 << 17, 256, 128, 1)),
          ((3, 512, 2, 64), BF, (1 << 17, 256, 64, 2)), ((3, 500, 2, 64), BF, None)],
    "v": [((3, 512, 2, 64), BF, (1 << 17, 256, 64, 1)), ((3, 512, 1, 64), BF, None), ((3, 512, 2, 64), F32, None)],
    "n": [((2,), I32, None), ((3,), F32, None), ((3,), I32, (2,)), ((3, 1), I32, None)],
    "start": [((2,), I32, None), ((3,), torch.int64, None), ((3,), I32, (2,))],
    "off": [((2,), I32, None), ((3,), torch.int64, None), ((3,), I32, (2,))],
    "ck": [((3, 512, 2, 64), U8, None), ((3, 512, 2, 64), torch.int8, None), ((3, 512, 2, 64), E4, (1 << 17, 256, 128, 1)), ((3, 512, 2, 32), E4, None)],
    "cv": [((3, 512, 2, 64), E4, (1 << 17, 256, 64, 1)), ((3, 512, 1, 64), E4, None), ((3, 512, 2, 64), torch.int8, None)],
    "ke": [((3, 512, 2), torch.int8, None), ((3, 2, 512), I32, None), ((3, 2, 512), torch.int8, (2048, 1024, 2))],
    "ve": [((3, 2, 511), torch.int8, None), ((3, 2, 512), torch.int8, (2048, 1024, 1)), ((3, 2, 512), U8, None)],
    "out": [((3, 4, 64), F32, None), ((3, 4, 64), BF, (512, 64, 1)), ((2, 4, 64), BF, None)],
    "qkv": [((3, 500), BF, None), ((3, 512), F32, None), ((3, 512), BF, (1, 3))],
    "gain": [((32,), BF, None), ((64,), F32, None), ((64,), BF, (2,))],
}


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_that_do_not_fit_are_refused(here, name):
    call, used = CALLS[name]
    for x in used.split():
        for shape, dtype, strides in WRONG[x]:
            if x == "start" and shape == (2,) and name in ("attn_prefill", "attn_prefill8", "cache8_read"):
                continue      # there it gives the number of sequences
            a = args()
            a[x] = Here(shape, dtype, strides)
            with pytest.raises((ValueError, TypeError)):
                call(a, None)
    assert not here.calls


@pytest.mark.parametrize("name", ["attn_decode", "attn_prefill", "attn_decode8", "attn_prefill8"])
def test_outputs_workspaces_and_windows_are_checked(here, name):
    call, _ = CALLS[name]
    for shape, dtype, strides in WRONG["out"]:
        with pytest.raises((ValueError, TypeError)):
            call(args(), None, out=Here(shape, dtype, strides))
    with pytest.raises(ValueError):
        call(args(), None, out=Here((3, 4, 64), BF, device=1))
    for ws in (Here((1 << 20,), U8, (2,)), Here((1 << 20,), U8, device=1)):
        with pytest.raises(ValueError):
            call(args(), None, workspace=ws)
    with pytest.raises(ValueError):
        call(args(), None, sinks=2**31)
    if name.endswith("8"):
        with pytest.raises(ValueError):
            call(args(), None, window=2**32 + 5)
    assert not here.calls


def test_more_sequences_than_the_cache_holds(here):
    a = args()
    for x, shape in (("q", (4, 4, 64)), ("n", (4,)), ("start", (4,)), ("off", (4,))):
        a[x] = Here(shape, a[x].dtype)
    with pytest.raises(ValueError):
        CALLS["attn_decode"][0](a, None)
    with pytest.raises(ValueError):
        kinv.cache8_read(cache(a), a["start"], a["n"], 10)
    with pytest.raises(ValueError):
        kinv.cache8_write(cache(a), Here((4, 10, 2, 64), BF), Here((4, 10, 2, 64), BF), a["start"], a["n"])
    with pytest.raises(ValueError):
        kinv.cache8_read(cache(a), a["start"], a["n"], k=a["k"])
    assert not here.calls


def test_records_name_a_window_only_where_there_is_one():
    from invariant_deterministic_gb300 import model, receipt
    sizes = dict(n_layers=2, d_model=256, n_q=4, n_kv=2, head_dim=64, ffn=512, vocab=512)
    plain, win = model.ModelShape(**sizes), model.ModelShape(**sizes, window=64, sinks=2)
    assert not {"window", "sinks"} & (set(receipt.model_identity(plain, 0)["shape"]) | set(receipt.settings_of(plain)))
    assert {"window": 64, "sinks": 2}.items() <= receipt.model_identity(win, 0)["shape"].items()
    assert model.ModelShape(**receipt.model_identity(win, 0)["shape"]) == win
    assert model.ModelShape(**receipt.model_identity(plain, 0)["shape"]) == plain
    assert receipt.settings_of(win, "int8")["cache"] == "int8" and "cache" not in receipt.settings_of(win)
