"""Attention with a sliding window and sinks, and over the 8-bit cache: against
the fp64 oracle, against each other's bits, and in the places where it can go
wrong (lengths around the splits, hidden slots of NaN, other batches, chunkings,
streams and graphs).

What is asked of the bits: attention over an 8-bit cache = attention over the
cache read back; a decode step = a one-row prefill; a row = the same row in any
batch or chunk; a window that hides nothing = no window."""
import numpy as np
import pytest
import torch

from helpers import assert_close, assert_same_bits, ensure_lib, f64, gpu, synth
from oracle import window as owin

pytestmark = gpu

HEADS = [(32, 8, 128), (4, 2, 64), (8, 1, 128), (2, 2, 64), (4, 2, 128), (8, 1, 64)]
I32 = dict(dtype=torch.int32, device="cuda")
NAN = float("nan")


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def i32(v):
    return torch.tensor(v, **I32)


def keys(shape, seed):
    """Keys or values of uneven loudness."""
    x = synth.normal_bf16(shape, 1.0, seed, "cuda")
    return x * torch.exp2(torch.randint(-3, 3, shape[:-1] + (1,), generator=synth.gen(seed + 7, "cuda"), device="cuda").to(torch.bfloat16))


def cache8(kinv, k, v, fmt):
    bsz, slots, hkv, d = k.shape
    c = kinv.Cache8.empty(bsz, slots, hkv, d, fmt)
    kinv.cache8_write(c, k, v, i32([0] * bsz), i32([slots] * bsz))
    return c, kinv.cache8_read(c, i32([0] * bsz), i32([slots] * bsz), slots)


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 255, 256, 257, 400, 511, 512, 513, 700, 768, 1000, 1023, 1024, 1025, 1100]
WINDOWS = [(1, 0), (1, 1), (16, 0), (64, 3), (255, 0), (256, 4), (257, 0), (300, 256), (300, 257), (512, 513), (700, 1), (5000, 9)]


# ------------------------------------------------------------ sliding window
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 3), (256, 300), (300, 0)])
def test_window_decode_against_the_oracle(kinv, hq, hkv, d, window, sinks):
    lens = [0, 1, 63, 64, 65, 256, 300, 556, 557, 700]
    k, v = keys((len(lens), 700, hkv, d), 60), keys((len(lens), 700, hkv, d), 61)
    q = synth.normal_bf16((len(lens), hq, d), 1.0, 62, "cuda")
    out = kinv.attn_decode(q, k, v, i32(lens), window=window, sinks=sinks)
    for b, n in enumerate(lens):
        ref = owin.row(f64(q[b]), f64(k[b]), f64(v[b]), n - 1, window, sinks)
        assert_close(f64(out[b]), ref, f"length {n}") if n else None
    assert (out[0] == 0).all() and kinv.last_device_status() == 0


@pytest.mark.parametrize("hq,hkv,d", HEADS[:4])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_decode_equals_prefill_and_full_attention_where_nothing_hides(kinv, hq, hkv, d, window, sinks):
    k, v = keys((1, 1100, hkv, d), 70).expand(len(LENS), -1, -1, -1), keys((1, 1100, hkv, d), 71).expand(len(LENS), -1, -1, -1)
    q = synth.normal_bf16((len(LENS), hq, d), 1.0, 72, "cuda")
    out = kinv.attn_decode(q, k, v, i32(LENS), window=window, sinks=sinks)
    full = kinv.attn_decode(q, k, v, i32(LENS))
    for b, n in enumerate(LENS):
        if n <= window + sinks or n <= window:
            assert_same_bits(out[b], full[b], f"length {n}")
        if n:
            one = kinv.attn_prefill(q[b: b + 1], k[:1], v[:1], i32([n - 1]), i32([1]), i32([0]), 1, n, window=window, sinks=sinks)
            assert_same_bits(one[0], out[b], f"prefill row {n - 1}")
    assert kinv.last_device_status() == 0


@pytest.mark.parametrize("hq,hkv,d", HEADS[:4])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 0), (64, 3), (256, 4), (300, 280), (600, 1)])
def test_window_prefill_rows_are_decode_steps_in_any_chunking(kinv, hq, hkv, d, window, sinks):
    n = 900
    k, v = keys((1, n, hkv, d), 80), keys((1, n, hkv, d), 81)
    q = synth.normal_bf16((n, hq, d), 1.0, 82, "cuda")

    def run(p0, rows):
        return kinv.attn_prefill(q[p0: p0 + rows], k, v, i32([p0]), i32([rows]), i32([0]), rows, p0 + rows, window=window, sinks=sinks)

    whole = run(0, n)
    for chunk in (7, 129, 512):
        parts = torch.cat([run(p, min(chunk, n - p)) for p in range(0, n, chunk)])
        assert_same_bits(parts, whole, f"chunks of {chunk}")
    rows = [0, 1, 39, 40, 255, 256, 300, 556, 580, 899]
    dec = kinv.attn_decode(q[rows], k.expand(len(rows), -1, -1, -1), v.expand(len(rows), -1, -1, -1), i32([r + 1 for r in rows]),
                           window=window, sinks=sinks)
    assert_same_bits(whole[rows], dec, "decode steps")
    for r in (300, 899):
        assert_close(f64(whole[r]), owin.row(f64(q[r]), f64(k[0]), f64(v[0]), r, window, sinks), f"row {r}")
    assert kinv.last_device_status() == 0


def test_window_prefill_of_ragged_sequences(kinv):
    hq, hkv, d, window, sinks = 32, 8, 128, 100, 2
    n, start = [5, 0, 300, 1, 64], [0, 10, 100, 650, 255]
    off = [3, 8, 8, 308, 309]
    rows = 380
    k, v = keys((5, 700, hkv, d), 90), keys((5, 700, hkv, d), 91)
    q = synth.normal_bf16((rows, hq, d), 1.0, 92, "cuda")
    out = torch.full_like(q, 7.0)
    kinv.attn_prefill(q, k, v, i32(start), i32(n), i32(off), 300, 700, out=out, window=window, sinks=sinks)
    assert (out[:3] == 7).all() and (out[373:] == 7).all()
    for b in range(5):
        if n[b]:
            one = kinv.attn_prefill(q[off[b]: off[b] + n[b]], k[b: b + 1], v[b: b + 1], i32([start[b]]), i32([n[b]]), i32([0]), n[b],
                                    start[b] + n[b], window=window, sinks=sinks)
            assert_same_bits(out[off[b]: off[b] + n[b]], one, f"sequence {b}")
    assert kinv.last_device_status() == 0


@pytest.mark.parametrize("bad", [NAN, float("inf"), torch.finfo(torch.bfloat16).min])
def test_what_hidden_slots_hold_does_not_matter(kinv, bad):
    hq, hkv, d, window, sinks = 8, 1, 128, 200, 5
    lens = [1000, 600, 210, 700]
    k, v = keys((4, 1024, hkv, d), 100), keys((4, 1024, hkv, d), 101)
    q = synth.normal_bf16((4, hq, d), 1.0, 102, "cuda")
    ref = kinv.attn_decode(q, k, v, i32(lens), window=window, sinks=sinks)
    k2, v2 = k.clone(), v.clone()
    for b, n in enumerate(lens):
        for t in (k2, v2):
            t[b, sinks: n - window] = bad
            t[b, n:] = bad
    assert_same_bits(kinv.attn_decode(q, k2, v2, i32(lens), window=window, sinks=sinks), ref, "decode")
    # a chunk of rows: what is hidden from all of them
    qs = synth.normal_bf16((50, hq, d), 1.0, 103, "cuda")
    args = (i32([900]), i32([50]), i32([0]), 50, 950)
    ref = kinv.attn_prefill(qs, k[:1], v[:1], *args, window=window, sinks=sinks)
    k2, v2 = k[:1].clone(), v[:1].clone()
    for t in (k2, v2):
        t[0, sinks: 901 - window] = bad
        t[0, 950:] = bad
    assert_same_bits(kinv.attn_prefill(qs, k2, v2, *args, window=window, sinks=sinks), ref, "prefill")


def test_window_with_every_cache_shape_of_a_batch(kinv):
    """A row's bits in other batches, at other slots, and in a cache of other strides."""
    hq, hkv, d, window, sinks = 4, 2, 64, 333, 7
    lens = synth.uniform_int(40, 0, 2000, 110).tolist()
    k, v = keys((40, 2000, hkv, d), 111), keys((40, 2000, hkv, d), 112)
    q = synth.normal_bf16((40, hq, d), 1.0, 113, "cuda")
    out = kinv.attn_decode(q, k, v, i32(lens), window=window, sinks=sinks)
    perm = torch.randperm(40, generator=synth.gen(114), ).cuda()
    wide_k, wide_v = (torch.full((40, 2100, hkv + 2, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wide_k[:, :2000, :hkv], wide_v[:, :2000, :hkv] = k[perm], v[perm]
    other = kinv.attn_decode(q[perm], wide_k[:, :, :hkv], wide_v[:, :, :hkv], i32(lens)[perm].contiguous(), window=window, sinks=sinks)
    assert_same_bits(other, out[perm], "permuted, other strides")
    assert kinv.last_device_status() == 0


@pytest.mark.parametrize("length", [-1, 701])
def test_window_lengths_outside_the_cache_give_zeros(kinv, length):
    k, v = keys((2, 700, 2, 64), 120), keys((2, 700, 2, 64), 121)
    q = synth.normal_bf16((2, 4, 64), 1.0, 122, "cuda")
    out = kinv.attn_decode(q, k, v, i32([length, 300]), window=50, sinks=1)
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
    assert (out[0] == 0).all() and not (out[1] == 0).all()
    c, _ = cache8(kinv, k, v, "int8")
    out8 = kinv.attn_decode8(q, c, i32([length, 300]))
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
    assert (out8[0] == 0).all() and not (out8[1] == 0).all()


# ------------------------------------------------------------ the 8-bit cache
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_decode8_has_the_bits_of_the_cache_read_back(kinv, hq, hkv, d, fmt):
    k, v = keys((len(LENS), 1100, hkv, d), 130), keys((len(LENS), 1100, hkv, d), 131)
    q = synth.normal_bf16((len(LENS), hq, d), 1.0, 132, "cuda")
    c, (k16, v16) = cache8(kinv, k, v, fmt)
    assert_same_bits(kinv.attn_decode8(q, c, i32(LENS)), kinv.attn_decode(q, k16, v16, i32(LENS)), "no window")
    assert_same_bits(kinv.attn_decode8(q, c, i32(LENS), scale=0.31), kinv.attn_decode(q, k16, v16, i32(LENS), scale=0.31), "scale")
    for window, sinks in WINDOWS:
        assert_same_bits(kinv.attn_decode8(q, c, i32(LENS), window=window, sinks=sinks),
                         kinv.attn_decode(q, k16, v16, i32(LENS), window=window, sinks=sinks), f"window {window}, sinks {sinks}")
    assert kinv.last_device_status() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("k_loud,v_loud,q_loud", [(0, 0, 0), (20, 0, -20), (-30, 0, 30), (0, 40, 0), (0, -60, 0), (0, 90, 0), (10, 30, -5)])
def test_decode8_at_every_loudness(kinv, fmt, k_loud, v_loud, q_loud):
    """Scales far from 1, and values of very different loudness beside each other."""
    hq, hkv, d, n = 8, 1, 128, 520
    k, v = keys((1, n, hkv, d), 140), keys((1, n, hkv, d), 141)
    k, v = k * 2.0 ** k_loud, v * 2.0 ** v_loud
    v = v * torch.exp2(torch.randint(-25, 25, (1, n, 1, 1), generator=synth.gen(142, "cuda"), device="cuda").to(torch.bfloat16))
    q = synth.normal_bf16((1, hq, d), 1.0, 143, "cuda") * 2.0 ** q_loud
    c, (k16, v16) = cache8(kinv, k, v, fmt)
    for n in (520, 256, 100):
        assert_same_bits(kinv.attn_decode8(q, c, i32([n])), kinv.attn_decode(q, k16, v16, i32([n])), f"length {n}")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d", HEADS[:4])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
def test_prefill8_has_the_bits_of_the_cache_read_back(kinv, hq, hkv, d, fmt, window, sinks):
    n, start, off = [70, 0, 200, 1], [0, 5, 412, 699], [0, 70, 70, 270]
    k, v = keys((4, 700, hkv, d), 150), keys((4, 700, hkv, d), 151)
    q = synth.normal_bf16((271, hq, d), 1.0, 152, "cuda")
    c, (k16, v16) = cache8(kinv, k, v, fmt)
    args = (i32(start), i32(n), i32(off), 200, 700)
    ws = torch.full((kinv.attn_prefill8_workspace(4, 271, hq, hkv, d, 700) // 2,), NAN, dtype=torch.bfloat16, device="cuda")
    out = kinv.attn_prefill8(q, c, *args, workspace=ws, window=window, sinks=sinks)
    # a window of all 700 keys hides nothing
    assert_same_bits(out, kinv.attn_prefill(q, k16, v16, *args, window=window or 700, sinks=sinks), "prefill")
    r, p = 70 + 199, 412 + 199
    dec = kinv.attn_decode8(q[r: r + 1], c.sequences(2, 3), i32([p + 1]), window=window, sinks=sinks)
    assert_same_bits(dec[0], out[r], "decode == prefill")
    assert kinv.last_device_status() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode8_hidden_and_marked_slots(kinv, fmt):
    hq, hkv, d, n = 32, 8, 128, 700
    k, v = keys((1, 800, hkv, d), 160), keys((1, 800, hkv, d), 161)
    q = synth.normal_bf16((1, hq, d), 1.0, 162, "cuda")
    c, _ = cache8(kinv, k, v, fmt)
    ref = kinv.attn_decode8(q, c, i32([n]), window=300, sinks=2)
    for t in (c.k, c.v):     # any bytes where nothing is visible
        t.view(torch.uint8)[:, 2:400] = 0xFF
        t.view(torch.uint8)[:, n:] = 0x7F
    for t in (c.k_exp, c.v_exp):
        t[:, :, 2:400] = -128
        t[:, :, n:] = -128
    assert_same_bits(kinv.attn_decode8(q, c, i32([n]), window=300, sinks=2), ref, "hidden slots")
    # a marked key or value makes its kv head's rows NaN, and no other's
    c.k_exp[0, 3, 500] = -128
    c.v_exp[0, 6, 699] = -128
    out = kinv.attn_decode8(q, c, i32([n]), window=300, sinks=2)
    bad = torch.isnan(out[0]).view(8, 4 * d).all(1).tolist()
    assert bad == [g in (3, 6) for g in range(8)]
    good = [h for h in range(hq) if h // 4 not in (3, 6)]
    assert_same_bits(out[0, good], ref[0, good], "the other heads")


@pytest.mark.parametrize("what", ["nan", "inf"])
def test_decode8_with_infinite_queries(kinv, what):
    q = synth.normal_bf16((2, 4, 64), 1.0, 170, "cuda")
    q[0, 1, 3] = NAN if what == "nan" else float("inf")
    k, v = keys((2, 300, 2, 64), 171), keys((2, 300, 2, 64), 172)
    c, (k16, v16) = cache8(kinv, k, v, "e4m3")
    a, b = kinv.attn_decode8(q, c, i32([300, 300])), kinv.attn_decode(q, k16, v16, i32([300, 300]))
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert_same_bits(torch.nan_to_num(a), torch.nan_to_num(b), "the rest")


def test_decode8_in_other_batches_and_strides(kinv):
    hq, hkv, d = 4, 2, 64
    lens = synth.uniform_int(40, 0, 3000, 180).tolist()
    k, v = keys((40, 3000, hkv, d), 181), keys((40, 3000, hkv, d), 182)
    q = synth.normal_bf16((40, hq, d), 1.0, 183, "cuda")
    c, (k16, v16) = cache8(kinv, k, v, "e4m3")
    out = kinv.attn_decode8(q, c, i32(lens))
    assert_same_bits(out, kinv.attn_decode(q, k16, v16, i32(lens)), "whole batch")
    perm = torch.randperm(40, generator=synth.gen(184)).cuda()
    wide = [torch.full((41, 3016, hkv + 3, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    exps = [torch.full((41, hkv + 1, 3016), 99, dtype=torch.int8, device="cuda") for _ in range(2)]
    for w, t in zip(wide + exps, c.tensors):
        if t.dim() == 4:
            w[:40, :3000, :hkv] = t.view(torch.uint8)[perm]
        else:
            w[:40, :hkv, :3000] = t[perm]
    c2 = kinv.Cache8(*(w[:40, :3000, :hkv].view(torch.float8_e4m3fn) for w in wide), *(e[:40, :hkv, :3000] for e in exps))
    assert_same_bits(kinv.attn_decode8(q[perm], c2, i32(lens)[perm].contiguous()), out[perm], "permuted, other strides")
    for b in (0, 17):
        one = kinv.attn_decode8(q[b: b + 1], c.sequences(b, b + 1), i32([lens[b]]))
        assert_same_bits(one[0], out[b], "alone")


def test_long_contexts(kinv):
    hq, hkv, d, n = 32, 8, 128, 40000
    k, v = keys((2, n, hkv, d), 190), keys((2, n, hkv, d), 191)
    q = synth.normal_bf16((2, hq, d), 1.0, 192, "cuda")
    lens = i32([n, 33333])
    for fmt in ("e4m3", "int8"):
        c, (k16, v16) = cache8(kinv, k, v, fmt)
        assert_same_bits(kinv.attn_decode8(q, c, lens), kinv.attn_decode(q, k16, v16, lens), fmt)
        assert_same_bits(kinv.attn_decode8(q, c, lens, window=20000, sinks=1000),
                         kinv.attn_decode(q, k16, v16, lens, window=20000, sinks=1000), fmt + " window")


# ------------------------------------------- few and many splits, far addresses
@pytest.mark.parametrize("splits", range(1, 10))
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 2, 64), (8, 1, 64)])
def test_few_and_many_sequences_of_few_splits(kinv, hq, hkv, d, splits):
    """Up to eight splits a small batch is one launch and a large one is not: the same
    bits, and those of attn_decode, for empty, short and out-of-range sequences too."""
    n = splits * 256 - 9
    lens = ([n, 1, 0, n - 1, max(n - 256, 0), 257 if n > 257 else 2] + synth.uniform_int(74, 0, n, 230 + splits).tolist())[:80]
    k, v = keys((80, n, hkv, d), 231), keys((80, n, hkv, d), 232)
    q = synth.normal_bf16((80, hq, d), 1.0, 233, "cuda")
    full = kinv.attn_decode(q, k, v, i32(lens))
    assert_same_bits(kinv.attn_decode(q, k, v, i32(lens), window=n), full, "a window of every key, large batch")
    assert_same_bits(kinv.attn_decode(q[:6], k[:6], v[:6], i32(lens[:6]), window=n), full[:6], "a window of every key, small batch")
    for window, sinks in ((max(n - 256, 1), 1), (40, 3)):
        many = kinv.attn_decode(q, k, v, i32(lens), window=window, sinks=sinks)
        for b in (0, 2, 77):
            assert_same_bits(kinv.attn_decode(q[b: b + 3], k[b: b + 3], v[b: b + 3], i32(lens[b: b + 3]), window=window, sinks=sinks),
                             many[b: b + 3], f"window {window}, small batch")
    for fmt in ("e4m3", "int8"):
        c, (k16, v16) = cache8(kinv, k, v, fmt)
        for window, sinks in ((0, 0), (max(n - 256, 1), 1)):
            ref = kinv.attn_decode(q, k16, v16, i32(lens), window=window, sinks=sinks)
            assert_same_bits(kinv.attn_decode8(q, c, i32(lens), window=window, sinks=sinks), ref, fmt + " large batch")
            for b in (0, 3):
                assert_same_bits(kinv.attn_decode8(q[b: b + 3], c.sequences(b, b + 3), i32(lens[b: b + 3]), window=window, sinks=sinks),
                                 ref[b: b + 3], fmt + " small batch")
        assert kinv.last_device_status() == 0
        c.v_exp[1, 0, 0] = -128
        out = kinv.attn_decode8(q[:3], c.sequences(0, 3), i32([n, 1, n + 1]))
        assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
        assert torch.isnan(out[1].view(hkv, -1)[0]).all() and (out[2] == 0).all() and not torch.isnan(out[0]).any()
    out = kinv.attn_decode(q[:2], k[:2], v[:2], i32([-1, n + 1]), window=40, sinks=3)
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG and (out == 0).all()


def test_sequences_more_than_two_gigabytes_apart(kinv):
    hq, hkv, d, n, far = 4, 2, 64, 600, 2**31 + 16 * 12345
    k, v = keys((3, n, hkv, d), 240), keys((3, n, hkv, d), 241)
    q = synth.normal_bf16((3, hq, d), 1.0, 242, "cuda")
    near, (k16, v16) = cache8(kinv, k, v, "e4m3")
    codes = [torch.empty(2 * far + n * hkv * d, dtype=torch.uint8, device="cuda").as_strided((3, n, hkv, d), (far, hkv * d, d, 1)) for _ in range(2)]
    exps = [torch.empty(3, hkv, n, dtype=torch.int8, device="cuda") for _ in range(2)]
    c = kinv.Cache8(*(t.view(torch.float8_e4m3fn) for t in codes), *exps)
    zero, full = i32([0] * 3), i32([n] * 3)
    kinv.cache8_write(c, k, v, zero, full)
    for a, b in zip(kinv.cache8_read(c, zero, full, n), (k16, v16)):
        assert_same_bits(a, b, "written and read")
    lens = i32([n, 300, n - 1])
    want = kinv.attn_decode(q, k16, v16, lens, window=400, sinks=3)
    assert_same_bits(kinv.attn_decode8(q, c, lens, window=400, sinks=3), want, "decode8")
    args = (i32([n - 1, 299, n - 2]), i32([1, 1, 1]), i32([0, 1, 2]), 1, n)
    assert_same_bits(kinv.attn_prefill8(q, c, *args, window=400, sinks=3), want, "prefill8")
    wide = [torch.empty(2 * far + n * hkv * d, dtype=torch.bfloat16, device="cuda").as_strided((3, n, hkv, d), (far, hkv * d, d, 1)) for _ in range(2)]
    kinv.cache8_read(c, zero, full, k=wide[0], v=wide[1])
    assert_same_bits(kinv.attn_decode(q, *wide, lens, window=400, sinks=3), want, "decode, bf16")
    assert_same_bits(kinv.attn_prefill(q, *wide, *args, window=400, sinks=3), want, "prefill, bf16")
    qkv = synth.normal_bf16((3, (hq + 2 * hkv) * d), 1.0, 243, "cuda")
    qs = [torch.empty_like(q) for _ in range(2)]
    for to, cc in zip(qs, (c, near)):
        kinv.rope_append8(qkv, to, cc, i32([0, 1, 2]), i32([599, 0, 77]), hq, hkv, d, 1e4)
    assert_same_bits(qs[0], qs[1], "q")
    for a, b in zip(kinv.cache8_read(c, zero, full, n), kinv.cache8_read(near, zero, full, n)):
        assert_same_bits(a, b, "appended")
    assert kinv.last_device_status() == 0


def test_prefill8_with_a_workspace_of_more_than_2_31_numbers(kinv):
    hq, hkv, d, bsz, n = 8, 8, 128, 36, 60000
    c = kinv.Cache8.empty(bsz, n, hkv, d, "int8")
    for b in (0, 35):
        x = keys((1, n, hkv, d), 250 + b)
        kinv.cache8_write(c.sequences(b, b + 1), x, x, i32([0]), i32([n]))
    q = synth.normal_bf16((bsz, hq, d), 1.0, 252, "cuda")
    out = kinv.attn_prefill8(q, c, i32([n - 1] * bsz), i32([1] * bsz), i32(list(range(bsz))), 1, n)
    assert_same_bits(out, kinv.attn_decode8(q, c, i32([n] * bsz)), "prefill8 == decode8")
    assert kinv.last_device_status() == 0


# --------------------------------------------------- a step, streams and graphs
def _step(kinv, c, s, window, sinks, ws=None):
    """Append the step's rows and attend, as a decode step does."""
    kinv.rope_append8(s["qkv"], s["q"], c, s["seq"], s["pos"], 8, 2, 64, 1e4)
    return kinv.attn_decode8(s["q"], c, s["len"], out=s["out"], workspace=ws, window=window, sinks=sinks)


def _inputs(step, seed=200):
    pos = torch.tensor([300, 5, 255, 511], **I32) + step
    return dict(qkv=synth.normal_bf16((4, 12 * 64), 1.0, seed + step, "cuda"), seq=torch.arange(4, **I32), pos=pos, len=pos + 1,
                q=torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda"), out=torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda"))


def _filled(kinv):
    k, v = keys((4, 600, 2, 64), 210), keys((4, 600, 2, 64), 211)
    return cache8(kinv, k, v, "e4m3")[0]


def test_captured_steps_equal_eager_ones(kinv):
    """Steps of append and attention replayed from a graph on new rows, two captured
    graphs with a workspace each, in turn."""
    want = []
    c = _filled(kinv)
    for t in range(3):
        want.append(_step(kinv, c, _inputs(t), 100, 2).clone())
    c = _filled(kinv)
    s = _inputs(0)
    graphs = []
    for _ in range(2):
        ws = torch.empty(kinv.attn_decode8_workspace(4, 8, 64, 600, 100, 2), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(kinv, c, s, 100, 2, ws)
        graphs.append((g, ws))
    for t in range(3):
        new = _inputs(t)
        for name in ("qkv", "pos", "len"):
            s[name].copy_(new[name])
        graphs[t % 2][0].replay()
        assert_same_bits(s["out"], want[t], f"step {t}")
    assert kinv.last_device_status() == 0


def test_steps_on_two_streams(kinv):
    want = []
    for w in (0, 64):
        want.append(_step(kinv, _filled(kinv), _inputs(0), w, 1).clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches, ins = [_filled(kinv) for _ in range(2)], [_inputs(0) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, c, s, w in zip(streams, caches, ins, (0, 64)):
            with torch.cuda.stream(st):
                _step(kinv, c, s, w, 1)
    torch.cuda.synchronize()
    for s, w in zip(ins, want):
        assert_same_bits(s["out"], w, "two streams")


def test_calls_on_a_named_stream(kinv):
    """stream= allocates from, runs on and holds memory for the named stream."""
    c = _filled(kinv)
    s = _inputs(0)
    want = _step(kinv, c, s, 90, 1).clone()
    x = keys((4, 50, 2, 64), 220)
    start, n = i32([1, 2, 3, 4]), i32([50, 7, 0, 33])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = kinv.attn_decode8(s["q"], c, s["len"], window=90, sinks=1, stream=side)
    k16, v16 = kinv.cache8_read(c, i32([0] * 4), i32([600] * 4), 600, stream=side)
    side.synchronize()
    assert_same_bits(out, want, "decode8")
    win = kinv.attn_decode(s["q"], k16, v16, s["len"], window=90, sinks=1, stream=side)
    args = (i32([299]), i32([2]), i32([0]), 2, 301)
    pre = kinv.attn_prefill(s["q"][:2].contiguous(), k16[:1], v16[:1], *args, window=90, sinks=1, stream=side)
    pre8 = kinv.attn_prefill8(s["q"][:2].contiguous(), c.sequences(0, 1), *args, window=90, sinks=1, stream=side)
    kinv.cache8_write(c, x, x, start, n, stream=side)
    side.synchronize()
    assert_same_bits(win, want, "decode")
    assert_same_bits(pre, pre8, "prefill")
    back = kinv.cache8_read(c, start, n, 50)[0]
    ref = cache8(kinv, x, x, "e4m3")[1][0]
    for b, m in enumerate([50, 7, 0, 33]):
        assert_same_bits(back[b, :m], ref[b, :m], "written")
    assert kinv.last_device_status() == 0


# ------------------------------------------- short chunks over many splits
FEW = [  # query heads, kv heads, D; rows of each sequence; their first positions; window, sinks
    ((32, 8, 128), [1], [8000], 0, 0), ((32, 8, 128), [33], [3000], 0, 0), ((32, 8, 128), [64], [5000], 700, 300),
    ((32, 8, 128), [128], [2100], 4000, 1), ((32, 8, 128), [0, 5, 32, 1], [10, 2500, 1000, 0], 0, 0),
    ((4, 2, 64), [100, 0, 64, 1, 65, 100], [0, 5, 1900, 1999, 1000, 255], 0, 0), ((4, 2, 64), [130, 7], [1500, 2000], 900, 4),
    ((8, 1, 128), [16, 17, 300], [1, 2000, 1500], 0, 0), ((8, 1, 128), [16, 17, 190], [1, 2000, 1500], 0, 0), ((8, 1, 64), [64] * 9, list(range(100, 1900, 200)), 1000, 0), ((2, 2, 64), [300], [1700], 0, 0),
    ((4, 4, 128), [1, 128], [1279, 4000], 1200, 600), ((32, 8, 128), [17, 3], [600, 0], 0, 0), ((4, 2, 64), [70], [500], 600, 1),
]


@pytest.mark.parametrize("heads,n,start,window,sinks", FEW, ids=str)
def test_short_chunks_spread_over_the_gpu_keep_their_bits(kinv, heads, n, start, window, sinks):
    hq, hkv, d = heads
    slots = max(a + b for a, b in zip(n, start)) + 9
    rows, bsz = sum(n) + 3, len(n)
    off = [2 + sum(n[:i]) for i in range(bsz)]
    k, v = keys((bsz, slots, hkv, d), 260), keys((bsz, slots, hkv, d), 261)
    q = synth.normal_bf16((rows, hq, d), 1.0, 262, "cuda")
    args = (i32(start), i32(n), i32(off), max(n), slots)
    big = window or slots + 1
    need = kinv.attn_prefill_window_workspace(bsz, max(n), hq, hkv, d, slots, big, sinks)
    tiles = -(-max(n) // (128 * hkv // hq)) * hkv * bsz
    assert (need > 0) == (tiles <= 38)       # more tiles stay whole
    out = torch.full_like(q, 7.0)
    ws = torch.full((max(need, 16) // 4,), NAN, dtype=torch.float32, device="cuda")
    kinv.attn_prefill(q, k, v, *args, out=out, workspace=ws, window=big, sinks=sinks)
    small = torch.empty(max(need - 16, 16), dtype=torch.uint8, device="cuda")     # too small: a block per tile
    whole = torch.full_like(q, 7.0)
    kinv.attn_prefill(q, k, v, *args, out=whole, workspace=small, window=big, sinks=sinks)
    assert_same_bits(out, whole, "spread == whole tiles")
    assert (out[:2] == 7).all() and (out[rows - 1:] == 7).all()
    for b in range(bsz):
        for i in sorted({0, n[b] // 2, n[b] - 1}) if n[b] else []:
            dec = kinv.attn_decode(q[off[b] + i: off[b] + i + 1], k[b: b + 1], v[b: b + 1], i32([start[b] + i + 1]), window=window, sinks=sinks)
            assert_same_bits(out[off[b] + i], dec[0], f"row {i} of sequence {b}")
    for fmt in ("e4m3", "int8"):
        c, (k16, v16) = cache8(kinv, k, v, fmt)
        got = torch.full_like(q, 7.0)
        kinv.attn_prefill8(q, c, *args, out=got, window=window, sinks=sinks)
        want = torch.full_like(q, 7.0)
        kinv.attn_prefill(q, k16, v16, *args, out=want, workspace=small, window=big, sinks=sinks)
        assert_same_bits(got, want, fmt)
    assert kinv.last_device_status() == 0


def test_short_chunks_with_numbers_outside_their_bounds_and_hidden_slots(kinv):
    """A sequence that breaks a bound is left out and reported; NaN where no row sees it;
    an infinite score stays with its rows."""
    hq, hkv, d, slots = 8, 1, 128, 3000
    k, v = keys((4, slots, hkv, d), 270), keys((4, slots, hkv, d), 271)
    q = synth.normal_bf16((20, hq, d), 1.0, 272, "cuda")
    good = (i32([2000, 2990, 1500, 100]), i32([5, 5, 5, 5]), i32([0, 5, 10, 15]), 5, slots)
    ref = kinv.attn_prefill(q, k, v, *good, window=1300, sinks=2)
    for t in (k, v):
        t[0, 2: 2001 - 1300] = NAN
        t[0, 2005:] = NAN
    out = torch.full_like(q, 7.0)
    kinv.attn_prefill(q, k, v, i32([2000, 2996, 1500, -1]), i32([5, 5, 6, 5]), i32([0, 5, 10, 15]), 5, slots, out=out, window=1300, sinks=2)
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
    assert (out[5:] == 7).all()
    assert_same_bits(out[:5], ref[:5], "the sequence that is left")
    kinv.attn_prefill(q, k, v, i32([2000, 2990, 1500, 100]), i32([5] * 4), i32([0, 16, 10, 15]), 5, slots, out=out, window=1300, sinks=2)
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG     # rows 16 .. 20 of 20
    assert_same_bits(out[10:15], ref[10:15], "another")


def test_short_chunks_on_two_streams_and_in_a_graph(kinv):
    hq, hkv, d, slots = 32, 8, 128, 4000
    k, v = keys((1, slots, hkv, d), 280), keys((1, slots, hkv, d), 281)
    c, _ = cache8(kinv, k, v, "int8")
    qs = [synth.normal_bf16((16, hq, d), 1.0, 282 + i, "cuda") for i in range(3)]
    args = (i32([3900]), i32([16]), i32([0]), 16, slots)
    want = [kinv.attn_prefill8(q, c, *args, window=3000, sinks=4) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, st in enumerate(streams):
            got.append((i, kinv.attn_prefill8(qs[i], c, *args, window=3000, sinks=4, stream=st)))
    torch.cuda.synchronize()
    for i, o in got:
        assert_same_bits(o, want[i], "two streams")
    q = qs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = kinv.attn_prefill8(q, c, *args, window=3000, sinks=4)
    for i in (2, 1, 0):
        q.copy_(qs[i])
        g.replay()
        assert_same_bits(o, want[i], "replayed")
