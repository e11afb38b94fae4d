"""What Decoder.score refuses before anything is launched (no GPU)."""
import types

import pytest
import torch

from invariant_deterministic_gb300 import kinv, model


@pytest.fixture
def dec(monkeypatch):
    def launched(*a, **kw):
        raise AssertionError("a kernel was given what score cannot score")
    monkeypatch.setattr(kinv, "embed", launched)
    d = model.Decoder.__new__(model.Decoder)
    d.B, d.Lmax, d.max_rows, d.dev = 2, 100, 16, torch.device("cpu")
    d.s, d.w = types.SimpleNamespace(vocab=50), {"embed": None}
    return d


class OnDevice:
    """A tensor that says it is on a CUDA device."""

    def __init__(self, t):
        self.t, self.is_cuda = t, True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, at):
        return OnDevice(self.t[at])


@pytest.mark.parametrize("tokens,error", [
    (torch.arange(9, dtype=torch.int32), ValueError),                          # host memory
    (OnDevice(torch.arange(9)), TypeError),                                    # 64-bit ids read as pairs of 32
    (OnDevice(torch.arange(18, dtype=torch.int32)[::2]), ValueError),          # every other id
    (OnDevice(torch.arange(18, dtype=torch.int32).view(9, 2)), ValueError),
    (OnDevice(torch.tensor(5, dtype=torch.int32)), ValueError),
])
def test_tokens_that_cannot_be_scored(dec, tokens, error):
    with pytest.raises(error):
        dec.score(0, tokens)
