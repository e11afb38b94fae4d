"""The 8-bit key/value cache on the GPU: codes and exponents against the oracle's
(equal bytes), reading back, and what the calls leave alone."""
import numpy as np
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth
from oracle import bf16 as obf, cache8 as o8, rope as orope
from oracle.rmsnorm import rmsnorm_f64

pytestmark = gpu

HEADS = [(32, 8, 128), (4, 2, 64), (8, 1, 128), (2, 2, 64)]
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def junk_cache(kinv, batch, slots, hkv, d, fmt, seed=900):
    """A cache whose slots hold something already."""
    c = kinv.Cache8.empty(batch, slots, hkv, d, fmt)
    g = synth.gen(seed, "cuda")
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(torch.randint(0, 127, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (c.k_exp, c.v_exp):
        t.copy_(torch.randint(-9, 3, t.shape, generator=g, device="cuda", dtype=torch.int8))
    return c


def loud(shape, seed):
    """bf16 vectors of very different loudness, some of zeros."""
    x = synth.normal_bf16(shape, 1.0, seed, "cuda")
    g = synth.gen(seed + 1, "cuda")
    e = torch.randint(-30, 30, shape[:-1] + (1,), generator=g, device="cuda")
    x = (x.float() * torch.exp2(e.float())).to(torch.bfloat16)
    x[torch.rand(shape[:-1], generator=g, device="cuda") < 0.05] = 0
    return x


def expect(x, fmt):
    codes, E = o8.quantise(synth.bits(x), fmt)
    return codes, E


def rotated_range(x, pos, base, gain, eps):
    """fp64 rotated heads x [T][H][D] -> (least, most) that fp32 arithmetic may give
    before the rounding to bf16.  An fp32 rotation of a pair (a, b), each with a
    relative error r1 from the norm, and sin and cos with errors r2, is off by at
    most (r1 + r2 + 2 u) (|a| + |b|) with u = 2^-24; r1 <= 11 u (a sum of 64 to 128
    squares by chains of eight and four pair sums, the sum with eps, root, reciprocal
    and two products; half of what is before the root), r2 <= 2 u (one rounding of
    a value that is right to 2^-27)."""
    y = obf.to_f64(synth.bits(x))
    if gain is not None:
        y = rmsnorm_f64(y, obf.to_f64(synth.bits(gain)), eps)
    half = y.shape[-1] // 2
    off = 16 * 2.0 ** -24 * (np.abs(y[..., :half]) + np.abs(y[..., half:]))
    off = np.concatenate([off, off], -1)
    z = orope.rope_f64(y, pos, base)
    return z - off, z + off


def held(codes, E, fmt):
    return o8.values(codes, E, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("rows", [1, 7, 130, 513])
def test_append_holds_the_codes_of_the_rotated_rows(kinv, hq, hkv, d, fmt, rows):
    """Values exactly; a key's code is that of some number that fp32 arithmetic may
    give (the exponent too), and the nominal one but for a few next to a border."""
    bsz, slots = 3, 400
    ld = (hq + 2 * hkv) * d + 16
    qkv = loud((rows, ld // 8, 8), 11).view(rows, ld)[:, :(hq + 2 * hkv) * d]
    places = torch.randperm(bsz * slots, generator=synth.gen(12))[:rows]
    seq, pos = (places // slots).to(**I32), (places % slots).to(**I32)
    qn = synth.normal_bf16((d,), 1.0, 13, "cuda") if rows != 7 else None
    kn = synth.normal_bf16((d,), 1.0, 14, "cuda") if rows != 7 else None
    q = torch.full((rows, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    c = junk_cache(kinv, bsz, slots, hkv, d, fmt)
    before = [raw(t).copy() for t in c.tensors]
    kinv.rope_append8(qkv, q, c, seq, pos, hq, hkv, d, 1e4, qn, kn)
    assert kinv.last_device_status() == 0
    heads = qkv.reshape(rows, hq + 2 * hkv, d)
    b, p = seq.long().cpu().numpy(), pos.long().cpu().numpy()
    lo, hi = rotated_range(heads[:, :hq], p, 1e4, qn, 1e-6)
    got = obf.to_f64(synth.bits(q))
    assert (obf.round_f64(lo) <= got).all() and (got <= obf.round_f64(hi)).all()
    after = [raw(t) for t in c.tensors]
    codes, E = expect(heads[:, hq + hkv:], fmt)
    assert np.array_equal(after[1][b, p], codes) and np.array_equal(after[3][b, :, p], E.view(np.uint8))
    # keys
    lo, hi = rotated_range(heads[:, hq: hq + hkv], p, 1e4, kn, 1e-6)
    mid, Em = o8.quantise(obf.from_f64((lo + hi) / 2), fmt)
    gc, gE = after[0][b, p], after[2][b, :, p].view(np.int8)
    least = np.maximum(np.maximum(lo, -hi), 0)          # |x| is at least this
    E_lo, E_hi = o8.exponent(obf.round_f64(least), fmt), o8.exponent(obf.round_f64(np.maximum(np.abs(lo), np.abs(hi))), fmt)
    assert ((E_lo <= gE) & (gE <= E_hi)).all()
    val, step = held(gc, gE, fmt), 2.0 ** gE.astype(np.float64)[..., None]
    for bound, sign in ((obf.round_f64(lo), 1.0), (obf.round_f64(hi), -1.0)):   # rounding to a code is monotone
        top = o8.LIMIT[fmt]
        y = np.clip(bound / step, -top, top)
        if fmt == "int8":
            r = np.rint(y)
        else:
            r = torch.from_numpy(y.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
        assert (sign * (val / step - r) >= 0).all()
    assert np.mean(val != held(mid, Em, fmt)) <= 1e-3 + 3 / gc.size   # (codes 0 and -0 stand for one value)
    # nothing else was written
    for now, was in zip(after, before):
        if now.ndim == 4:
            now[b, p] = was[b, p]
        else:
            now[b, :, p] = was[b, :, p]
        assert np.array_equal(now, was)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_infinities_nan_and_the_largest_numbers(kinv, fmt):
    hq, hkv, d, slots = 2, 2, 64, 8
    inf, nan, top = float("inf"), float("nan"), 3.3895313892515355e38
    qkv = synth.normal_bf16((6, 6 * d), 1.0, 5, "cuda").view(6, 6, d)
    qkv[0, 2, 5], qkv[1, 4, 63], qkv[2, 5, 0], qkv[3, 4, 1], qkv[4, 5, 7] = inf, nan, -inf, top, -top
    qkv[5, 4] = 2.0 ** -133
    qkv = qkv.view(6, -1)
    seq, pos = torch.zeros(6, **I32), torch.arange(1, 7, **I32)
    q = torch.empty(6, hq, d, dtype=torch.bfloat16, device="cuda")
    c = kinv.Cache8.empty(1, slots, hkv, d, fmt)
    kinv.rope_append8(qkv, q, c, seq, pos, hq, hkv, d, 1e4)
    got = kinv.cache8_read(c, torch.zeros(1, **I32), torch.tensor([slots], **I32), slots)
    # the key of row 0's head 0 holds an infinity: marked; the others are finite
    assert c.k_exp[0, 0, 1] == -128 and not c.k[0, 1, 0].view(torch.uint8).any() and torch.isfinite(got[0][0, 2:7]).all()
    codes, E = expect(qkv.view(6, 6, d)[:, 4:], fmt)
    assert np.array_equal(raw(c.v[0, 1:7]), codes) and np.array_equal(c.v_exp[0, :, 1:7].cpu().numpy(), E.T)
    want, back = torch.from_numpy(o8.values(codes, E, fmt)).to(torch.bfloat16), got[1][0, 1:7].cpu()
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(back), torch.nan_to_num(want)) and not torch.isinf(back).any()
    assert torch.isnan(got[1][0, 2, 0]).all() and torch.isnan(got[0][0, 1, 0]).all()


def test_append_leaves_out_rows_outside_the_cache(kinv):
    hq, hkv, d = 4, 2, 64
    qkv = synth.normal_bf16((6, 8 * d), 1.0, 21, "cuda")
    seq, pos = torch.tensor([0, 2, -1, 1, 0, 1], **I32), torch.tensor([3, 3, 3, 50, -1, 49], **I32)
    c = junk_cache(kinv, 2, 50, hkv, d, "e4m3")
    before = [raw(t).copy() for t in c.tensors]
    q = torch.full((6, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    kinv.rope_append8(qkv, q, c, seq, pos, hq, hkv, d, 1e4)
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG and kinv.last_device_status() == 0
    assert [bool((q[r] == 9).all()) for r in range(6)] == [False, True, True, True, True, False]
    for t, was in zip(c.tensors, before):
        now = raw(t)
        if t.dim() == 4:
            now[0, 3], now[1, 49] = was[0, 3], was[1, 49]
        else:
            now[0, :, 3], now[1, :, 49] = was[0, :, 3], was[1, :, 49]
        assert np.array_equal(now, was)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d", HEADS + [(16, 16, 64), (3, 3, 128)])
def test_write_and_read_back(kinv, hq, hkv, d, fmt):
    bsz, n, slots = 4, 100, 150
    lens, starts = [100, 0, 33, 1], [50, 20, 3, 149]
    wide = loud((bsz, n, hkv + 1, d), 31)
    k, v = wide[:, :, :hkv], loud((bsz, n, hkv + 1, d), 33)[:, :, :hkv]   # tokens further apart than their heads
    start, length = torch.tensor(starts, **I32), torch.tensor(lens, **I32)
    c = junk_cache(kinv, bsz + 1, slots, hkv, d, fmt)
    want = [raw(t).copy() for t in c.tensors]
    kinv.cache8_write(c, k, v, start, length)
    for i, x in ((0, k), (1, v)):
        codes, E = expect(x, fmt)
        for b in range(bsz):
            want[i][b, starts[b]: starts[b] + lens[b]] = codes[b, :lens[b]]
            want[2 + i][b, :, starts[b]: starts[b] + lens[b]] = E[b, :lens[b]].T.view(np.uint8)
    for t, w, name in zip(c.tensors, want, ("k", "v", "k_exp", "v_exp")):
        assert np.array_equal(raw(t), w), name
    out = [torch.full((bsz, n, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kinv.cache8_read(c, start, length, k=out[0], v=out[1])
    for i in (0, 1):
        val = o8.values(want[i], want[2 + i].view(np.int8).transpose(0, 2, 1), fmt)
        ref = torch.full((bsz, n, hkv, d), 5.0, dtype=torch.bfloat16)
        for b in range(bsz):
            ref[b, :lens[b]] = torch.from_numpy(val[b, starts[b]: starts[b] + lens[b]]).to(torch.bfloat16)
        assert_same_bits(out[i].cpu(), ref, "read back")
    assert kinv.last_device_status() == 0
    # writing what was read back changes nothing
    before = [kinv.cache8_read(c, start, length, n)[i].clone() for i in (0, 1)]
    kinv.cache8_write(c, before[0], before[1], start, length)
    after = kinv.cache8_read(c, start, length, n)
    for b in range(bsz):
        for i in (0, 1):
            assert_same_bits(after[i][b, :lens[b]], before[i][b, :lens[b]], "written again")


@pytest.mark.parametrize("start,length", [(-1, 4), (147, 4), (0, -1), (0, 9), (2**31 - 1, 4)])
def test_ranges_outside_the_bounds_are_left_out(kinv, start, length):
    c = junk_cache(kinv, 2, 150, 2, 64, "int8")
    before = [raw(t).copy() for t in c.tensors]
    x = synth.normal_bf16((2, 8, 2, 64), 1.0, 41, "cuda")
    s, n = torch.tensor([start, 5], **I32), torch.tensor([length, 3], **I32)
    kinv.cache8_write(c, x, x, s, n)
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
    for t, was in zip(c.tensors, before):
        now = raw(t)
        sub = (1, slice(5, 8)) if t.dim() == 4 else (1, slice(None), slice(5, 8))
        assert not np.array_equal(now[sub], was[sub])
        now[sub] = was[sub]
        assert np.array_equal(now, was)
    out = [torch.full((2, 8, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kinv.cache8_read(c, s, n, k=out[0], v=out[1])
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
    for o in out:
        assert (o[0] == 5).all() and (o[1, 3:] == 5).all() and not (o[1, :3] == 5).all()


def test_calls_without_rows_or_tokens(kinv):
    c = junk_cache(kinv, 2, 16, 2, 64, "e4m3")
    before = [raw(t).copy() for t in c.tensors]
    none = torch.zeros(0, **I32)
    kinv.rope_append8(torch.zeros(0, 6 * 64, dtype=torch.bfloat16, device="cuda"),
                      torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda"), c, none, none, 2, 2, 64, 1e4)
    x = torch.zeros(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    two = torch.zeros(2, **I32)
    kinv.cache8_write(c, x, x, two, two)
    kinv.cache8_read(c, two, two, 0)
    assert kinv.last_device_status() == 0
    assert all(np.array_equal(raw(t), was) for t, was in zip(c.tensors, before))


def test_a_cache_past_two_to_the_31_bytes(kinv):
    """Slots behind 2^31 bytes of codes, one sequence's and the last one's."""
    hkv, d, slots = 8, 128, 2_200_000
    c = kinv.Cache8.empty(1, slots, hkv, d, "e4m3")
    x = synth.normal_bf16((1, 70, hkv, d), 1.0, 51, "cuda")
    start, length = torch.tensor([slots - 70], **I32), torch.tensor([70], **I32)
    kinv.cache8_write(c, x, x, start, length)
    codes, E = expect(x, "e4m3")
    assert np.array_equal(raw(c.k[:, slots - 70:]), codes) and np.array_equal(raw(c.v[:, slots - 70:]), codes)
    assert np.array_equal(c.k_exp[:, :, slots - 70:].cpu().numpy(), E.transpose(0, 2, 1))
    assert not c.k[:, :slots - 70].view(torch.uint8).any()
    k, v = kinv.cache8_read(c, start, length, 70)
    ref = torch.from_numpy(o8.values(codes, E, "e4m3")).to(torch.bfloat16)
    assert_same_bits(k.cpu(), ref, "k")
    q = synth.normal_bf16((1, 8, d), 1.0, 52, "cuda")
    # the last 70 keys, against a cache that begins at a split's border behind 2^31 bytes
    base = (slots - 70) // 256 * 256 - 512
    near = kinv.Cache8(c.k[:, base:], c.v[:, base:], c.k_exp[:, :, base:], c.v_exp[:, :, base:])
    far = kinv.attn_decode8(q, c, torch.tensor([slots], **I32), window=70)
    assert_same_bits(far, kinv.attn_decode8(q, near, torch.tensor([slots - base], **I32), window=70), "the last keys")
    assert far.any()
    assert kinv.last_device_status() == 0
