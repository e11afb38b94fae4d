"""The scratch of prefill over an 8-bit cache is sized by the window and the chunk."""
import os
import shutil

import pytest
import torch

from helpers import assert_same_bits, gpu


@pytest.fixture(scope="module")
def kinv():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from invariant_deterministic_gb300 import build, kinv
    build.build()
    return kinv


PART = 128 * (128 + 2) * 4   # a tile's partial of one split, heads of 128


def test_a_call_of_known_rows_and_window_needs_what_it_uses(kinv):
    back = 131072 * 8 * 128 * 4
    size = lambda rows, **kw: kinv.attn_prefill8_workspace(1, rows, 32, 8, 128, 131072, **kw)  # noqa: E731
    assert size(4096) == back + 32 * 512 * PART                                    # any window, any chunk
    assert size(4096, max_q_len=4096) == back                                      # tiles stay whole
    assert size(4096, max_q_len=4096, window=4096, sinks=4) == back
    assert size(128, max_q_len=128) == back + 32 * 512 * PART
    assert size(128, max_q_len=128, window=4096, sinks=4) == back + 32 * 19 * PART  # 4,096 + 31 keys: 18 splits, and one of sinks
    assert size(16, max_q_len=16) == back + 8 * 512 * PART
    assert size(16, max_q_len=2**31 - 1) == back + 8 * 512 * PART                  # rows of the call, whatever the bound
    assert kinv.attn_prefill8_workspace(3, 0, 32, 8, 128, 1000, max_q_len=5) == 0
    # no call of fewer rows or of a window needs more than the size without a bound
    for rows in (1, 33, 100, 128, 129, 1000):
        for window, sinks in ((0, 0), (1, 0), (300, 9), (131072, 0)):
            assert size(rows, max_q_len=rows, window=window, sinks=sinks) <= size(rows)


def _decoder(kinv, window, max_chunk, max_batch=2, max_len=1500):
    from invariant_deterministic_gb300 import model as M
    shape = M.ModelShape(n_layers=2, d_model=256, n_q=4, n_kv=2, head_dim=64, ffn=512, vocab=512, window=window, sinks=3 if window else 0)
    return M.Decoder(shape, M.random_weights(shape, seed=1, device="cuda"), max_batch=max_batch, max_len=max_len, max_chunk=max_chunk,
                     cache="e4m3")


@gpu
@pytest.mark.parametrize("window", [0, 300])
def test_a_decoder_holds_the_scratch_of_its_chunks(kinv, window):
    decode = kinv.attn_decode8_workspace(2, 4, 64, 1500, window, 3 if window else 0)
    plain = _decoder(kinv, window, 0)
    assert plain.ws.numel() == max(decode, 256)
    chunked = _decoder(kinv, window, 200)
    back = 1500 * 2 * 64 * 4
    splits = (300 + 63 + 254) // 256 + 1 + 1 if window else 6
    assert chunked.ws.numel() == max(decode, back + 2 * 4 * splits * 128 * (64 + 2) * 4)   # four tiles of 64 rows, two kv heads
    # prompts go through either, with the same bits
    tokens = torch.randint(0, 512, (900,), dtype=torch.int32, device="cuda")
    ends = [dec.prefill(1, tokens) for dec in (plain, chunked)]
    assert_same_bits(ends[0], ends[1], "a prompt in chunks of 2 and of 200 rows")
    for a, b in zip(plain.kv8, chunked.kv8):
        for x, y in zip(a.tensors, b.tensors):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert kinv.last_device_status() == 0
