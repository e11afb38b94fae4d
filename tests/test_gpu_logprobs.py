"""kinv_logprobs on the GPU against the fp64 oracle, row invariance, and the
rows where it can go wrong.

Tolerances.  A term 2^a of S has the error of ex2.approx (2 ulp: 2^-22) and of
its argument a = fl(fl(x - m) log2e): three roundings of at most 2^-24 relative
(difference, product, the constant), times ln 2 |a| <= ln V + ... as a relative
error of the term; weighted by the terms themselves the sum of |a| ln 2 p is at
most ln V <= 14, so 42 * 2^-24.  Every term passes at most 17 + 5 additions in
its unit and 63 + 5 in the fold (90 * 2^-24), so S is off by at most (4 + 42 +
90) 2^-24 = 8.2e-6 relative and ln S by that much absolutely, plus one rounding
of ln S and two of the differences (2^-23 relative).  The entropy ln S - ln 2
T / S carries T's and S's relative errors (8.2e-6 each, T's terms have one more
rounding) times ln 2 |T| / S <= ln S <= 12 for these rows: 8.2e-6 (1 + 2 * 12)."""
import numpy as np
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth
from oracle import logprobs as olp

pytestmark = gpu
ATOL, RTOL, ENTROPY_ATOL = 8.2e-6, 2.0 ** -22, 2.1e-4


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def close(got, want, what, atol=ATOL):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= atol + RTOL * np.abs(want))
    assert ok.all(), f"{what}: {got[~ok][:4]} against {want[~ok][:4]}"


def check(kinv, x, ids, k, rows=None):
    """Every row of x (float64 copies of what the GPU holds) against the oracle."""
    lp, h, ti, tl = kinv.logprobs(x, ids, top_k=k)
    assert kinv.last_device_status() == 0
    xs = x.float().cpu().numpy().astype(np.float64)
    for r in range(x.shape[0]) if rows is None else rows:
        full, ent = olp.row(xs[r])
        close(h[r].item(), ent, f"entropy of row {r}", ENTROPY_ATOL)
        if ids is not None:
            i = ids[r].cpu().numpy()
            close(lp[r].cpu().numpy(), np.where(i < 0, 0.0, full[np.maximum(i, 0)]), f"row {r}")
        if k:
            want = olp.top(xs[r], k)
            assert ti[r].tolist() == want.tolist(), f"top ids of row {r}"
            close(tl[r].cpu().numpy(), full[want], f"top logprobs of row {r}")
    return lp, h, ti, tl


def logits(rows, v, seed, dtype=torch.float32, std=3.0):
    x = torch.randn(rows, v, generator=synth.gen(seed, "cuda"), device="cuda") * std
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [1, 2, 31, 32, 33, 511, 512, 513, 1000, 4096, 4097, 32000, 151936])
@pytest.mark.parametrize("rows", [1, 3])
def test_sizes(kinv, dtype, v, rows):
    x = logits(rows, v, v, dtype)
    ids = torch.randint(0, v, (rows, 3), generator=synth.gen(1)).to(torch.int32)
    ids[0, 1] = -1
    for k in sorted({0, 1, min(5, v), min(32, v)}):
        check(kinv, x, ids.cuda(), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows_have_the_bits_of_one(kinv, dtype):
    rows, v = 1300, 20011
    x = logits(rows, v + 13, 5, dtype)[:, :v]            # an odd row length: no 16-byte loads
    ids = torch.randint(0, v, (rows, 2), generator=synth.gen(2)).to(torch.int32).cuda()
    whole = check(kinv, x, ids, 20, rows=[0, 7, 1299])
    for r0, n in ((0, 1), (7, 1), (100, 3), (640, 70), (0, 160), (0, 303), (0, 305)):
        part = kinv.logprobs(x[r0: r0 + n], ids[r0: r0 + n], top_k=20)
        for a, b in zip(part, whole):
            assert_same_bits(a, b[r0: r0 + n], f"rows {r0} .. {r0 + n}")
    # the same rows where 16-byte loads apply, and at an odd address
    wide = torch.empty(rows, 20032, dtype=dtype, device="cuda")
    wide[:, :v] = x
    for a, b in zip(kinv.logprobs(wide[:, :v], ids, top_k=20), whole):
        assert_same_bits(a, b, "aligned rows")
    flat = torch.empty(rows * 20032 + 1, dtype=dtype, device="cuda")[1:].view(rows, 20032)
    flat.copy_(wide)
    for a, b in zip(kinv.logprobs(flat[:, :v], ids, top_k=20), whole):
        assert_same_bits(a, b, "rows at an odd address")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [1, 40, 1023, 1025, 8192])
def test_many_short_rows(kinv, dtype, v):
    """Rows that take one warp of a block each, the last block part empty."""
    rows, k = 2437, min(v, 32)
    x = logits(rows, v, v, dtype)
    ids = torch.randint(0, v, (rows, 2), generator=synth.gen(6)).to(torch.int32).cuda()
    whole = check(kinv, x, ids, k, rows=[0, 9, rows - 1])
    for r0, n in ((0, 1), (rows - 1, 1), (1000, 300)):
        for a, b in zip(kinv.logprobs(x[r0: r0 + n], ids[r0: r0 + n], top_k=k), whole):
            assert_same_bits(a, b[r0: r0 + n], f"rows {r0} .. {r0 + n}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [600, 20000])
def test_rows_where_it_can_go_wrong(kinv, dtype, v):
    inf, low = float("inf"), torch.finfo(dtype).min
    x = logits(16, v, 9, dtype)
    x[0] = 1.5                                            # all equal: the lowest ids, in order
    x[1] = -inf
    x[2] = float("nan")
    x[3, ::2] = float("nan")
    x[4] = -inf
    x[4, 300] = 2.0                                       # one possible id
    x[5, [5, 400]] = inf
    x[6] = low                                            # masks of the type's lowest value
    x[7] = low
    x[7, 411] = 3.0
    x[8] = torch.linspace(-20, 20, v).to(dtype).cuda()    # each id likelier than all before it
    x[9] = torch.linspace(20, -20, v).to(dtype).cuda()
    x[10] = 0.0
    x[10, 1::2] = -0.0                                    # equal to 0: ids decide
    x[11] *= 1e30
    x[12] *= 1e-30
    x[13, :] = -inf
    x[13, 7] = float("nan")
    x[14, 3] = torch.finfo(dtype).max
    x[15] = torch.randint(0, 3, (v,), generator=synth.gen(4)).to(dtype).cuda()   # many ties
    ids = torch.randint(0, v, (16, 4), generator=synth.gen(3)).to(torch.int32)
    ids[:, 0] = 300
    ids[3, 1] = 0
    ids[5] = torch.tensor([5, 400, 6, -3], dtype=torch.int32)
    ids[14, 1] = 3
    for k in (1, 20, 32):
        check(kinv, x, ids.cuda(), k)
    # the same rows in a batch that takes one block per row
    many = x.repeat(50, 1)
    alone = kinv.logprobs(x, ids.cuda(), top_k=32)
    for a, b in zip(kinv.logprobs(many, ids.repeat(50, 1).cuda(), top_k=32), alone):
        assert_same_bits(a[-16:], b, "in a large batch")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_maxima(kinv, dtype):
    """Maxima around 1e30 of either sign over ids far below them and masks."""
    inf, low = float("inf"), torch.finfo(dtype).min
    tops = (9.9e29, 1.01e30, -9.9e29, -1.01e30, 3e38, -3e38, 1e29, -1e29)
    x = torch.empty(len(tops), 3000, dtype=dtype, device="cuda")
    for r, m in enumerate(tops):
        below = [t for t in (-2e30, -2.1e30, low, -inf, float("nan"), m - abs(m) / 16) if not t >= m]
        x[r] = torch.tensor([below[i % len(below)] for i in range(3000)], dtype=torch.float64).to(dtype).cuda()
        x[r, [10, 2500]] = m                              # two ids share the row
    ids = torch.tensor([[10, 2500, 0, 1500]] * len(tops), dtype=torch.int32).cuda()
    check(kinv, x, ids, 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [700, 1030, 2060, 5000, 50001])
def test_any_alignment_gives_the_same_bits(kinv, dtype, v):
    """Rows at every offset from the 16-byte grid, with even and odd distances."""
    plain = logits(6, v, 21, dtype)
    ids = torch.randint(0, v, (6, 3), generator=synth.gen(5)).to(torch.int32).cuda()
    want = kinv.logprobs(plain, ids, top_k=20)
    for at in range(9):
        for pad in (0, 1, 2, 4):
            wide = torch.full((6, at + v + pad), float("nan"), dtype=dtype, device="cuda")
            wide[:, at: at + v] = plain
            for a, b in zip(kinv.logprobs(wide[:, at: at + v], ids, top_k=20), want):
                assert_same_bits(a, b, f"offset {at}, distance {at + v + pad}")
    assert kinv.last_device_status() == 0


def test_an_id_beyond_the_vocabulary_is_reported(kinv):
    x = logits(2, 700, 1)
    ids = torch.tensor([[0, 700], [2147483647, -2147483648]], **dict(dtype=torch.int32, device="cuda"))
    lp = kinv.logprobs(x, ids)[0]
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
    assert torch.isnan(lp[0, 1]) and torch.isnan(lp[1, 0]) and lp[1, 1] == 0 and torch.isfinite(lp[0, 0])


def test_two_streams_and_capture(kinv):
    x = logits(4, 151936, 2)
    ids = torch.randint(0, 151936, (4, 1), generator=synth.gen(3)).to(torch.int32).cuda()
    want = kinv.logprobs(x, ids, top_k=8)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(6):
        outs.append(kinv.logprobs(x, ids, top_k=8, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, want):
            assert_same_bits(a, b, "two streams")
    s = streams[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = kinv.logprobs(x, ids, top_k=8)
    for seed in (2, 6):
        x.copy_(logits(4, 151936, seed))
        g.replay()
        for a, b in zip(got, kinv.logprobs(x, ids, top_k=8)):
            assert_same_bits(a, b, "replayed")
