"""The 8-bit cache's calls in the launch plans of many rows and tokens, and the angles of
far positions and other bases."""
import numpy as np
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth
from oracle import bf16 as obf, cache8 as o8
from test_gpu_cache8 import HEADS, I32, expect, junk_cache, loud, raw, rotated_range

pytestmark = gpu


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# A block takes one row up to 4 an SM, then up to 16; more blocks than one wave from 64 an SM.
ROWS = {"two rows a block": lambda: 4 * sms() + 1, "a partial last block": lambda: 4 * sms() + 93, "a prompt chunk": lambda: 4096,
        "sixteen a block": lambda: 64 * sms(), "a second wave": lambda: 64 * sms() + 1, "two waves": lambda: 100 * sms() + 7}


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d", HEADS + [(7, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("plan", list(ROWS))
def test_append_of_many_rows_has_the_bits_of_a_row_a_block(kinv, hq, hkv, d, fmt, plan):
    rows = ROWS[plan]()
    width, slots = (hq + 2 * hkv) * d, 1 << 14
    qkv = loud((rows, width // 8, 8), 41).view(rows, width)
    g = synth.gen(42)
    places = torch.randperm(3 * slots, generator=g)[:rows]
    seq, pos = (places // slots).to(**I32), (places % slots).to(**I32)
    out_of_it = torch.rand(rows, generator=g) < 0.02
    seq[out_of_it.cuda()] = 3                       # rows outside the cache, left out
    qn, kn = (synth.normal_bf16((d,), 1.0, s, "cuda") if plan != "a prompt chunk" else None for s in (43, 44))
    got, want = junk_cache(kinv, 3, slots, hkv, d, fmt), junk_cache(kinv, 3, slots, hkv, d, fmt)
    q, q_want = (torch.full((rows, hq, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kinv.rope_append8(qkv, q, got, seq, pos, hq, hkv, d, 1e6, qn, kn)
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
    for r in range(0, rows, 300):
        e = min(rows, r + 300)
        kinv.rope_append8(qkv[r:e], q_want[r:e], want, seq[r:e], pos[r:e], hq, hkv, d, 1e6, qn, kn)
    kinv.last_device_status()
    assert_same_bits(q, q_want, "queries")
    assert (q[out_of_it.cuda()] == 3).all()
    for a, b, name in zip(got.tensors, want.tensors, ("k", "v", "k_exp", "v_exp")):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("rows", [9, 700])
@pytest.mark.parametrize("base,slots", [(0.05, 1 << 20), (1e4, 1 << 20), (1e6, 1 << 20), (1e4, 1 << 23)])
def test_append_at_far_positions(kinv, hq, hkv, d, fmt, rows, base, slots):
    """As near the oracle as at the first positions (a base below 1 / (2 pi) has
    frequencies above a turn a position)."""
    base = float(np.float32(base))                  # the argument's type
    g = synth.gen(51)
    pos = torch.unique(torch.exp2(torch.rand(4 * rows, generator=g, dtype=torch.float64) * np.log2(slots)).long() - 1)
    pos = pos[torch.randperm(len(pos), generator=g)][:rows - 2]
    pos = torch.cat([pos[pos < slots - 2], torch.tensor([slots - 1, slots - 2])]).to(**I32)
    rows = len(pos)
    qkv = loud((rows, (hq + 2 * hkv) * d // 8, 8), 52).view(rows, -1)
    qn, kn = synth.normal_bf16((d,), 1.0, 53, "cuda"), synth.normal_bf16((d,), 1.0, 54, "cuda")
    q = torch.full((rows, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    c = kinv.Cache8.empty(1, slots, hkv, d, fmt)
    kinv.rope_append8(qkv, q, c, torch.zeros(rows, **I32), pos, hq, hkv, d, base, qn, kn)
    assert kinv.last_device_status() == 0
    heads, p = qkv.view(rows, hq + 2 * hkv, d), pos.cpu().numpy()
    lo, hi = rotated_range(heads[:, :hq], p, base, qn, 1e-6)
    got = obf.to_f64(synth.bits(q))
    assert (obf.round_f64(lo) <= got).all() and (got <= obf.round_f64(hi)).all()
    at = pos.long()
    codes, E = expect(heads[:, hq + hkv:], fmt)
    assert np.array_equal(raw(c.v[0, at]), codes) and np.array_equal(raw(c.v_exp[0][:, at]).T, E.view(np.uint8))
    lo, hi = rotated_range(heads[:, hq: hq + hkv], p, base, kn, 1e-6)
    gE = c.k_exp[0][:, at].T.cpu().numpy()
    least = np.maximum(np.maximum(lo, -hi), 0)
    assert ((o8.exponent(obf.round_f64(least), fmt) <= gE)
            & (gE <= o8.exponent(obf.round_f64(np.maximum(np.abs(lo), np.abs(hi))), fmt))).all()
    val, step = o8.values(raw(c.k[0, at]), gE, fmt), 2.0 ** gE.astype(np.float64)[..., None]
    for bound, sign in ((obf.round_f64(lo), 1.0), (obf.round_f64(hi), -1.0)):
        y = np.clip(bound / step, -o8.LIMIT[fmt], o8.LIMIT[fmt])
        r = np.rint(y) if fmt == "int8" else torch.from_numpy(y.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
        assert (sign * (val / step - r) >= 0).all()


@pytest.mark.parametrize("base", [0.05, 1e4, 1e6])
def test_angles_are_right_to_more_than_fp32(kinv, base):
    """A query of ones and zeros comes out as the cosines and sines, in bf16 by way of fp32.
    Where an fp32 number is right to e before its rounding, it is rounded the other way
    for about 2 e / 2^-24 of the numbers in [1/2, 1), and two of 2^16 such changes change
    the bf16 number: at the e = 2^-28 that the series give at most 2^-18 of the numbers,
    with series in single floats (2^-24 and more) 2^-14."""
    base = float(np.float32(base))                  # the argument's type
    rows, d, slots = 1 << 18, 128, 1 << 20
    qkv = torch.zeros(rows, 3, d, dtype=torch.bfloat16, device="cuda")
    qkv[:, 0, : d // 2] = 1
    pos = torch.randperm(slots, generator=synth.gen(61))[:rows].to(**I32)
    q = torch.empty(rows, 1, d, dtype=torch.bfloat16, device="cuda")
    kinv.rope_append8(qkv.view(rows, -1), q, kinv.Cache8.empty(1, slots, 1, d), torch.zeros(rows, **I32), pos, 1, 1, d, base)
    assert kinv.last_device_status() == 0
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    wrong = 0
    for r in range(0, rows, 1 << 16):
        th = pos[r: r + (1 << 16), None].double() * base ** (-2.0 * i / d)
        want = torch.cat([torch.cos(th), torch.sin(th)], 1).float().to(torch.bfloat16)
        wrong += int((q[r: r + (1 << 16), 0] != want).sum())
    assert wrong <= rows * d * 2.0 ** -18


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_codes_of_a_prompt_chunk_against_64_bits(kinv, fmt):
    """4,096 rows of the large layer with norms.  About ten fp32 roundings leave an error of
    about 2^-24 of a number, so a bf16 number goes the other way for about 2 2^-24 / 2^-8
    of them (twice that for the smaller half of a binade, 2^-14 in all) and its code for
    less than a quarter of those (a code's step holds 16 of bf16's, or 2 to 2^7)."""
    rows, hq, hkv, d, base = 4096, 32, 8, 128, 1e6
    qkv = synth.normal_bf16((rows, (hq + 2 * hkv) * d), 1.0, 71, "cuda")
    qn, kn = (1 + 0.1 * synth.normal_bf16((d,), 1.0, s, "cuda").float() for s in (72, 73))
    qn, kn = qn.to(torch.bfloat16), kn.to(torch.bfloat16)
    pos = torch.arange(28000, 28000 + rows, **I32)
    q = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    c = kinv.Cache8.empty(1, 32768, hkv, d, fmt)
    kinv.rope_append8(qkv, q, c, torch.zeros(rows, **I32), pos, hq, hkv, d, base, qn, kn)
    assert kinv.last_device_status() == 0
    x = qkv.view(rows, hq + 2 * hkv, d).double()
    th = pos[:, None].double() * base ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
    cos, sin = torch.cos(th)[:, None], torch.sin(th)[:, None]

    def turned(h, gain):
        h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * gain.double()
        a, b = h[..., : d // 2], h[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)

    assert float((q != turned(x[:, :hq], qn)).double().mean()) <= 2.0 ** -14
    want = kinv.Cache8.empty(1, 32768, hkv, d, fmt)
    zero, n = torch.tensor([28000], **I32), torch.tensor([rows], **I32)
    kinv.cache8_write(want, turned(x[:, hq: hq + hkv], kn)[None], qkv.view(1, rows, -1, d)[:, :, hq + hkv:].contiguous(), zero, n)
    assert torch.equal(c.v.view(torch.uint8), want.v.view(torch.uint8)) and torch.equal(c.v_exp, want.v_exp)
    got, ref = (kinv.cache8_read(z, zero, n, rows)[0] for z in (c, want))
    assert float((got != ref).double().mean()) <= 2.0 ** -16


@pytest.mark.parametrize("hkv,d,fmt", [(2, 64, "e4m3"), (3, 128, "int8"), (8, 128, "e4m3")])
def test_write_and_read_of_32_tokens_a_block(kinv, hkv, d, fmt):
    bsz, n = 4, 16 * sms() + 77                     # 32 tokens a block from 608 blocks on
    lens, starts = [n, n - 31, 0, 1023], [11, 0, 5, n - 1000]
    slots = n + 40
    k, v = loud((bsz, n, hkv, d), 81), loud((bsz, n, hkv, d), 83)
    start, length = torch.tensor(starts, **I32), torch.tensor(lens, **I32)
    c = junk_cache(kinv, bsz, slots, hkv, d, fmt)
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
        for b in range(bsz):
            ref = torch.from_numpy(val[b, starts[b]: starts[b] + lens[b]]).to(torch.bfloat16)
            assert_same_bits(out[i][b, :lens[b]].cpu(), ref, "read back")
            assert (out[i][b, lens[b]:] == 5).all()
    assert kinv.last_device_status() == 0
