"""Prefill's rows behind several splits, every one of them, in the bits of the decode
step at their position."""
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth

pytestmark = gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def i32(v):
    return torch.tensor(v, **I32)


def uneven(shape, seed):
    x = synth.normal_bf16(shape, 1.0, seed, "cuda")
    loud = torch.randint(-3, 3, shape[:-1] + (1,), generator=synth.gen(seed + 7, "cuda"), device="cuda")
    return x * torch.exp2(loud.to(torch.bfloat16))


def decode_rows(kinv, q, k, v, first):
    """Rows q as decode steps at positions first .. of one sequence, 250 at a time."""
    out = torch.empty_like(q)
    for r in range(0, len(q), 250):
        m = min(250, len(q) - r)
        out[r: r + m] = kinv.attn_decode(q[r: r + m], k.expand(m, -1, -1, -1), v.expand(m, -1, -1, -1),
                                         i32(range(first + r + 1, first + r + m + 1)))
    return out


# 32, 64, 16 and 128 rows per tile
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 2, 64), (8, 1, 128), (2, 2, 64), (16, 2, 64), (16, 16, 128)])
@pytest.mark.parametrize("make", ["even", "uneven"])
def test_every_row_of_a_prompt_is_its_decode_step(kinv, hq, hkv, d, make):
    n = 2000
    keys = uneven if make == "uneven" else (lambda shape, seed: synth.normal_bf16(shape, 1.0, seed, "cuda"))
    k, v = keys((1, n, hkv, d), 20), keys((1, n, hkv, d), 21)
    q = synth.normal_bf16((n, hq, d), 1.0, 22, "cuda")
    whole = kinv.attn_prefill(q, k, v, i32([0]), i32([n]), i32([0]), n, n)
    assert_same_bits(whole, decode_rows(kinv, q, k, v, 0), "rows of one chunk")
    late = kinv.attn_prefill(q[900:], k, v, i32([900]), i32([n - 900]), i32([0]), n - 900, n)
    assert_same_bits(late, whole[900:], "a chunk behind 900 keys")
    assert kinv.last_device_status() == 0


def test_every_row_of_ragged_chunks_behind_long_contexts_is_its_decode_step(kinv):
    hq, hkv, d = 32, 8, 128
    start, n = [3000, 0, 1279, 700], [200, 1, 77, 513]
    off = [0, 200, 201, 278]
    k, v = uneven((4, 3200, hkv, d), 30), uneven((4, 3200, hkv, d), 31)
    q = synth.normal_bf16((sum(n), hq, d), 1.0, 32, "cuda")
    out = kinv.attn_prefill(q, k, v, i32(start), i32(n), i32(off), max(n), 3200)
    for b in range(4):
        dec = decode_rows(kinv, q[off[b]: off[b] + n[b]], k[b: b + 1], v[b: b + 1], start[b])
        assert_same_bits(out[off[b]: off[b] + n[b]], dec, f"sequence {b}")
    assert kinv.last_device_status() == 0
