"""Trees of drafted tokens on the GPU: a drafted row has the bits of the decode
step behind its path, against the fp64 oracle, at the edges of the 256-key
splits and 16-key steps; rotation and append; acceptance and the cache's move."""
import numpy as np
import pytest
import torch

from helpers import assert_close, assert_same_bits, ensure_lib, f64, gpu, synth
from oracle import bf16 as obf, tree as otree

pytestmark = gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def shape_parents(shape, n, seed=0):
    """Parents of a tree of n nodes."""
    g = synth.gen(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "star":
        return [-1] + [0] * (n - 1)
    if shape == "bushy":
        return [-1] + [r(i // 4, max(i // 4, i // 2 - 1)) if i > 1 else 0 for i in range(1, n)]
    if shape == "forest":  # several nodes follow the context itself
        return [-1 if i % 5 == 0 else r(max(0, i - 6), i - 1) for i in range(n)]
    raise ValueError(shape)


class Case:
    """Trees `parents[b]` behind `ctx[b]` cached keys."""

    def __init__(self, kinv, ctx, parents, hq, hkv, d, slots=None, seed=0, gap=0, pad_tok=0, poison=True):
        self.kinv, self.ctx, self.parents, self.hq, self.hkv, self.d = kinv, ctx, parents, hq, hkv, d
        B = len(ctx)
        n = [len(p) for p in parents]
        self.slots = slots or max(c + k for c, k in zip(ctx, n)) + 1
        self.off, at = [], gap
        for k in n:
            self.off.append(at)
            at += k + gap
        self.rows = max(at, 1)
        parent = torch.full((self.rows,), -7, dtype=torch.int32)   # rows of no sequence: never read
        for o, p in zip(self.off, parents):
            parent[o: o + len(p)] = torch.tensor(p, dtype=torch.int32)
        wide = hkv * d + pad_tok
        self.k = synth.normal_bf16((B, self.slots, wide), 1.0, seed + 1, "cuda")[..., : hkv * d].view(B, self.slots, hkv, d)
        self.v = synth.normal_bf16((B, self.slots, wide), 1.0, seed + 2, "cuda")[..., : hkv * d].view(B, self.slots, hkv, d)
        if poison:  # slots that hold nothing of the sequence
            for b in range(B):
                self.k[b, ctx[b] + n[b]:] = float("nan")
                self.v[b, ctx[b] + n[b]:] = float("nan")
        self.q = synth.normal_bf16((self.rows, hq, d), 1.0, seed + 3, "cuda")
        self.tree = kinv.Tree(torch.tensor(ctx, **I32), torch.tensor(n, **I32), torch.tensor(self.off, **I32),
                              parent.cuda(), max(max(n), 1), self.slots)

    def run(self, **kw):
        return self.kinv.attn_tree(self.q, self.k, self.v, self.tree, **kw)

    def decode(self, b):
        """Sequence b's rows as decode rows over the context and each path in order."""
        p = self.parents[b]
        if not p:
            return torch.empty(0, self.hq, self.d, dtype=torch.bfloat16, device="cuda")
        paths = [otree.path_of(p, i) for i in range(len(p))]
        lens = [self.ctx[b] + len(x) for x in paths]
        at = torch.zeros(len(p), max(lens), dtype=torch.int64)
        for i, x in enumerate(paths):
            at[i, : lens[i]] = torch.tensor(list(range(self.ctx[b])) + [self.ctx[b] + j for j in x])
        at = at.cuda()
        return self.kinv.attn_decode(self.q[self.off[b]: self.off[b] + len(p)].contiguous(), self.k[b][at].contiguous(),
                                     self.v[b][at].contiguous(), torch.tensor(lens, **I32))

    def check_bits(self, out, what=""):
        for b in range(len(self.ctx)):
            assert_same_bits(out[self.off[b]: self.off[b] + len(self.parents[b])], self.decode(b), f"{what} sequence {b}")


HEADS = [(32, 8, 128), (4, 2, 64), (8, 1, 128), (2, 2, 64), (8, 1, 64), (2, 2, 128), (4, 2, 128)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("shape", ["chain", "bushy", "star", "forest"])
def test_rows_have_the_bits_of_decode(kinv, hq, hkv, d, shape):
    # contexts around the steps of 16 and the splits of 256 keys, trees of 1 to 64 nodes
    ctx = [0, 1, 15, 16, 17, 200, 240, 255, 256, 257, 511, 700]
    n = [64, 1, 2, 3, 5, 64, 17, 33, 64, 31, 8, 13]
    c = Case(kinv, ctx, [shape_parents(shape, k, seed=i) for i, k in enumerate(n)], hq, hkv, d)
    out = c.run()
    assert kinv.last_device_status() == 0
    c.check_bits(out, shape)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 2, 64), (8, 1, 128), (2, 2, 64)])
def test_against_the_oracle(kinv, hq, hkv, d):
    ctx, shapes, n = [0, 37, 250, 600], ["bushy", "forest", "chain", "star"], [7, 20, 12, 3]
    c = Case(kinv, ctx, [shape_parents(s, k, seed=9) for s, k in zip(shapes, n)], hq, hkv, d, seed=20)
    out = c.run()
    for b in range(4):
        ref = otree.attention(synth.bits(c.q[c.off[b]: c.off[b] + n[b]]), synth.bits(c.k[b]), synth.bits(c.v[b]), ctx[b],
                              c.parents[b])
        assert_close(f64(out[c.off[b]: c.off[b] + n[b]]), obf.to_f64(ref), f"sequence {b}")


@pytest.mark.parametrize("n", [1, 4, 16, 32, 64])
def test_long_context(kinv, n):
    """Many splits; a tree whose pairs fill one and several tiles."""
    c = Case(kinv, [9001, 32000 - 64], [shape_parents("bushy", n, 3), shape_parents("chain", n)], 32, 8, 128, slots=32000, seed=40,
             poison=False)
    c.check_bits(c.run(), f"{n} nodes")


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_many_splits_with_every_head_layout(kinv, hq, hkv, d):
    """Contexts of several splits (enough of them for the tensor-core path, which
    deals the splits of all sequences out in equal runs), ragged trees, sequences
    without a whole split and without nodes in between."""
    ctx = [2600, 100, 0, 5000, 256, 511, 7000, 1023, 1024, 30, 4096, 255, 9000]
    n = [5, 64, 3, 0, 64, 1, 33, 40, 64, 8, 17, 2, 63]
    parents = [shape_parents(["bushy", "chain", "forest"][i % 3], k, i) if k else [] for i, k in enumerate(n)]
    c = Case(kinv, ctx, parents, hq, hkv, d, seed=50, gap=1, pad_tok=8)
    out = torch.full_like(c.q, 7.0)
    c.run(out=out)
    assert kinv.last_device_status() == 0
    c.check_bits(out, "many splits")


def test_batch_and_slot_invariance(kinv):
    parents = [shape_parents("bushy", k, k) for k in (5, 64, 1, 30)]
    ctx = [1000, 300, 0, 513]
    c = Case(kinv, ctx, parents, 32, 8, 128, seed=60)
    out = c.run()
    for b in (0, 1, 3):
        one = Case(kinv, [ctx[b]], [parents[b]], 32, 8, 128, slots=c.slots, seed=60)
        one.k, one.v = c.k[b: b + 1], c.v[b: b + 1]
        one.q = c.q[c.off[b]: c.off[b] + len(parents[b])].contiguous()
        assert_same_bits(one.run(), out[c.off[b]: c.off[b] + len(parents[b])], f"sequence {b} alone")
    # a node does not depend on the nodes that do not precede it: the first 20 of the 64 alone
    one = Case(kinv, [ctx[1]], [parents[1][:20]], 32, 8, 128, slots=c.slots, seed=60)
    one.k, one.v, one.q = c.k[1:2], c.v[1:2], c.q[c.off[1]: c.off[1] + 20].contiguous()
    assert_same_bits(one.run(), out[c.off[1]: c.off[1] + 20], "the first nodes of a tree")


@pytest.mark.parametrize("pad_tok,gap", [(0, 3), (8, 0), (64, 2)])
def test_strides_and_rows_of_no_sequence(kinv, pad_tok, gap):
    parents = [shape_parents("bushy", 9, 1), [], shape_parents("forest", 6, 2)]
    c = Case(kinv, [100, 50, 260], parents, 4, 2, 64, seed=80, gap=gap, pad_tok=pad_tok)
    out = torch.full_like(c.q, 7.0)
    c.run(out=out)
    c.check_bits(out, "padded strides")
    used = torch.zeros(c.rows, dtype=torch.bool)
    for o, p in zip(c.off, parents):
        used[o: o + len(p)] = True
    assert torch.all(out[~used.cuda()] == 7.0)
    assert kinv.last_device_status() == 0


def test_broken_trees_are_left_out_and_reported(kinv):
    parents = [shape_parents("bushy", 9, 1), shape_parents("chain", 6), shape_parents("star", 5)]
    good = Case(kinv, [100, 300, 20], parents, 4, 2, 64, seed=90, slots=310)
    want = good.run()

    def broken(index, value, which):
        t = [x.clone() for x in good.tree.tensors]
        t[which][index] = value
        return kinv.Tree(*t, good.tree.max_nodes, good.tree.max_kv)

    o = good.off[1]
    for tree in (broken(1, -1, 0), broken(1, 305, 0), broken(1, 2147483647, 0), broken(1, -1, 1), broken(1, 10, 1),
                 broken(1, -1, 2), broken(1, good.rows - 5, 2), broken(1, 2147483647, 2),
                 broken(o, 0, 3), broken(o + 3, 3, 3), broken(o + 3, 5, 3), broken(o + 5, -2, 3), broken(o + 1, 2147483647, 3)):
        out = torch.full_like(good.q, 7.0)
        kinv.attn_tree(good.q, good.k, good.v, tree, out=out)
        assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
        for b in (0, 2):
            assert_same_bits(out[good.off[b]: good.off[b] + len(parents[b])], want[good.off[b]: good.off[b] + len(parents[b])], "beside")
        assert torch.all(out[o: o + 6] == 7.0)
        k, v, q = good.k.clone(), good.v.clone(), torch.full_like(good.q, 7.0)
        qkv = synth.normal_bf16((good.rows, 8 * 64), 1.0, 5, "cuda")
        kinv.rope_append_tree(qkv, q, k, v, tree, 4, 2, 64, 1e4)
        assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
        assert torch.all(q[o: o + 6] == 7.0) and not torch.any(q[: o] == 7.0)
        assert_same_bits(k[1], good.k[1], "a left-out sequence's cache")
        tok = torch.zeros(good.rows, **I32)
        kv = torch.stack([good.k, good.v])[None].contiguous()
        before = kv.clone()
        cnt, path, _ = kinv.tree_accept(tree, tok, tok, kv, n_accepted=torch.full((3,), -5, **I32))
        assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
        assert cnt.tolist()[1] == -5 and cnt.tolist()[0] > 0 and cnt.tolist()[2] > 0
        assert_same_bits(kv[:, :, 1], before[:, :, 1], "a left-out sequence's cache")


def test_nothing_to_do(kinv):
    c = Case(kinv, [5, 9], [[], []], 4, 2, 64)
    out = torch.full_like(c.q, 7.0)
    c.run(out=out)
    assert torch.all(out == 7.0) and kinv.last_device_status() == 0
    cnt, path, tok = kinv.tree_accept(c.tree, torch.zeros(c.rows, **I32), torch.zeros(c.rows, **I32))
    assert cnt.tolist() == [0, 0] and path.tolist() == [[-1], [-1]] and tok.tolist() == [[-1], [-1]]


def test_infinite_and_nan_keys_stay_with_the_rows_that_see_them(kinv):
    parents = [[-1, 0, 0, 1, 2, 0]]
    c = Case(kinv, [30], parents, 4, 2, 64, seed=95)
    clean = c.run()
    for t, value in ((c.v, float("nan")), (c.v, float("inf")), (c.k, float("nan"))):
        keep = t.clone()
        t[0, 30 + 2] = value                      # node 2: seen by itself and node 4
        out = c.run()
        for i in (0, 1, 3, 5):
            assert_same_bits(out[i], clean[i], f"node {i}")
        c.check_bits(out, "rows that see it") if value != value and t is c.v else None
        t.copy_(keep)


def test_workspace_scale_and_streams(kinv):
    c = Case(kinv, [300, 20], [shape_parents("bushy", 40, 1), shape_parents("chain", 3)], 32, 8, 128, seed=100)
    want = c.run()
    need = kinv.attn_tree_workspace(c.tree, 32, 8, 128)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    assert_same_bits(c.run(workspace=ws[:need]), want, "a workspace of NaN bits")
    assert torch.all(ws[need:] == 0xFF)
    with pytest.raises(kinv.KinvError) as e:
        c.run(workspace=ws[: need - 1])
    assert e.value.status == kinv.ERR_WORKSPACE
    assert_same_bits(c.run(scale=float(1 / np.sqrt(128))), want, "the default scale given")
    # two calls at once on two streams, a workspace each
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(a if i % 2 else b):
            outs.append(c.run(workspace=ws[:need] if i % 2 else None))
    torch.cuda.synchronize()
    for o in outs:
        assert_same_bits(o, want, "two streams")


def test_captured_step_follows_the_trees_tensors(kinv):
    """One captured graph replayed with other trees, lengths and contents."""
    hq, hkv, d, slots, rows = 32, 8, 128, 900, 80
    B = 3
    t = [torch.zeros(B, **I32), torch.zeros(B, **I32), torch.zeros(B, **I32), torch.zeros(rows, **I32)]
    tree = kinv.Tree(*t, 64, slots)
    k, v = synth.normal_bf16((B, slots, hkv, d), 1.0, 1, "cuda"), synth.normal_bf16((B, slots, hkv, d), 1.0, 2, "cuda")
    qkv = synth.normal_bf16((rows, (hq + 2 * hkv) * d), 1.0, 3, "cuda")
    q, out = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kinv.attn_tree_workspace(tree, hq, hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        kinv.rope_append_tree(qkv, q, k, v, tree, hq, hkv, d, 1e6)
        kinv.attn_tree(q, k, v, tree, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for ctx, n in (([100, 0, 830], [10, 1, 64]), ([5, 255, 512], [64, 3, 0])):
        off = np.cumsum([0] + n[:-1]).tolist()
        parent = sum([shape_parents("bushy", x, 3) for x in n if x], [])
        for dst, src in zip(t, (ctx, n, off, parent)):
            dst[: len(src)].copy_(torch.tensor(src, dtype=torch.int32))
        qkv.copy_(synth.normal_bf16(tuple(qkv.shape), 1.0, sum(ctx), "cuda"))
        g.replay()
        got = out.clone(), q.clone(), k.clone()
        step()
        for a, b_ in zip(got, (out, q, k)):
            assert_same_bits(a, b_, "replayed against called")
    assert kinv.last_device_status() == 0


@pytest.mark.parametrize("hq,hkv,d,norm", [(32, 8, 128, True), (4, 2, 64, False), (8, 1, 128, False), (2, 2, 64, True)])
@pytest.mark.parametrize("big", [False, True])
def test_rope_append_tree_has_the_bits_of_rope_append(kinv, hq, hkv, d, norm, big):
    n = [64, 17, 1, 0, 40] * (5 if big else 1)       # more than 512 rows, and few
    ctx = [5, 0, 100, 7, 31] * (5 if big else 1)
    parents = [shape_parents(["bushy", "chain", "forest"][i % 3], x, i) for i, x in enumerate(n)]
    c = Case(kinv, ctx, parents, hq, hkv, d, seed=110, gap=1, poison=False)
    qkv = synth.normal_bf16((c.rows, (hq + 2 * hkv) * d + 8), 1.0, 7, "cuda")[:, : (hq + 2 * hkv) * d]
    gains = [(1 + 0.1 * torch.randn(d, generator=synth.gen(s))).to(torch.bfloat16).cuda() if norm else None for s in (1, 2)]
    q = torch.full((c.rows, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = c.k.clone(), c.v.clone()
    kinv.rope_append_tree(qkv, q, k, v, c.tree, hq, hkv, d, 1e6, *gains)
    assert kinv.last_device_status() == 0
    # every row through kinv_rope_append at its position, into a cache of its own
    seq, pos, row, slot = [], [], [], []
    for b, p in enumerate(parents):
        for i in range(len(p)):
            seq.append(b), row.append(c.off[b] + i), slot.append(ctx[b] + i)
            pos.append(ctx[b] + len(otree.path_of(p, i)) - 1)
    rows = torch.tensor(row).cuda()
    src = qkv[rows].contiguous()
    kr = torch.zeros(len(row), max(pos) + 1, hkv, d, dtype=torch.bfloat16, device="cuda")
    vr = torch.zeros_like(kr)
    qr = torch.empty(len(row), hq, d, dtype=torch.bfloat16, device="cuda")
    kinv.rope_append(src, qr, kr, vr, torch.arange(len(row), **I32), torch.tensor(pos, **I32), hq, hkv, d, 1e6, *gains)
    each = torch.arange(len(row)).cuda()
    assert_same_bits(q[rows], qr, "q")
    assert_same_bits(k[seq, slot], kr[each, torch.tensor(pos).cuda()], "keys")
    assert_same_bits(v[seq, slot], vr[each, torch.tensor(pos).cuda()], "values")
    k[seq, slot] = c.k[seq, slot]
    v[seq, slot] = c.v[seq, slot]
    assert_same_bits(k, c.k, "the other slots")
    assert_same_bits(v, c.v, "the other slots")
    others = torch.ones(c.rows, dtype=torch.bool)
    others[row] = False
    assert torch.all(q[others.cuda()] == 7.0)


@pytest.mark.parametrize("layers,hkv,d", [(3, 2, 64), (1, 8, 128), (36, 1, 128), (2, 1, 8)])
def test_accept_against_the_oracle(kinv, layers, hkv, d):
    ctx, n = [0, 11, 3, 20, 1, 2], [64, 9, 1, 0, 33, 64]
    shapes = ["chain", "bushy", "chain", "chain", "bushy", "forest"]
    parents = [shape_parents(s, k, i) if k else [] for i, (s, k) in enumerate(zip(shapes, n))]
    off = np.cumsum([2] + [k + 1 for k in n[:-1]]).tolist()
    rows = off[-1] + n[-1]
    slots = max(c + k for c, k in zip(ctx, n))
    g = synth.gen(3)
    tok = torch.randint(0, 4, (rows,), generator=g)      # few distinct tokens: equal siblings happen
    nxt = torch.randint(0, 4, (rows,), generator=g)
    parent = torch.full((rows,), 9, dtype=torch.int32)
    for o, p in zip(off, parents):
        parent[o: o + len(p)] = torch.tensor(p, dtype=torch.int32)
    tok[off[0]: off[0] + 64] = nxt[off[0]: off[0] + 64] = 1       # a chain that is taken whole: nothing moves
    tree = kinv.Tree(torch.tensor(ctx, **I32), torch.tensor(n, **I32), torch.tensor(off, **I32), parent.cuda(), 64, slots)
    kv = synth.normal_bf16((layers, 2, len(n), slots, hkv, d), 1.0, 4, "cuda")
    want_kv = kv.clone()
    cnt, path, out = kinv.tree_accept(tree, tok.to(torch.int32).cuda(), nxt.to(torch.int32).cuda(), kv)
    for b in range(len(n)):
        t, x = tok[off[b]: off[b] + n[b]].tolist(), nxt[off[b]: off[b] + n[b]].tolist()
        want = otree.accept(parents[b], t, x)
        assert cnt[b].item() == len(want)
        assert path[b].tolist() == want + [-1] * (64 - len(want))
        assert out[b].tolist() == [x[j] for j in want] + [-1] * (64 - len(want))
        for i, j in enumerate(want):
            want_kv[:, :, b, ctx[b] + i] = kv_slot(want_kv, b, ctx[b] + j)
    assert_same_bits(kv, want_kv, "cache")
    assert kinv.last_device_status() == 0
    # without a cache: the path alone
    again = kinv.tree_accept(tree, tok.to(torch.int32).cuda(), nxt.to(torch.int32).cuda())
    for a, b_ in zip(again, (cnt, path, out)):
        assert torch.equal(a, b_)


def kv_slot(kv, b, slot):
    return kv[:, :, b, slot].clone()


@pytest.mark.parametrize("n", [4, 64])
def test_caches_past_32_bits(kinv, n):
    """Slots 2.2 million elements apart: the last of a sequence's 1,000 lies past
    2^31 elements and 2^32 bytes, for a few nodes and for the tensor-core path."""
    hq, hkv, d, slots, tok = 32, 8, 128, 1000, 2_200_000
    base = torch.empty(2, slots, tok, dtype=torch.bfloat16, device="cuda")
    kv = base.as_strided((1, 2, 2, slots, hkv, d), (8, 4096, slots * tok, tok, d, 1))
    ctx = [990 - n, 800]
    parents = [shape_parents("bushy", n, 1), shape_parents("chain", n)]
    c = Case(kinv, ctx, parents, hq, hkv, d, slots=slots, seed=120, poison=False)
    kv[0, 0], kv[0, 1] = c.k, c.v
    qkv = synth.normal_bf16((c.rows, (hq + 2 * hkv) * d), 1.0, 7, "cuda")
    tok_, nxt = (synth.uniform_int(c.rows, 0, 2, s).to(torch.int32).cuda() for s in (8, 9))
    got = []
    for k, v in ((c.k, c.v), (kv[0, 0], kv[0, 1])):
        q = torch.zeros(c.rows, hq, d, dtype=torch.bfloat16, device="cuda")
        kinv.rope_append_tree(qkv, q, k, v, c.tree, hq, hkv, d, 1e6)
        got.append((q, kinv.attn_tree(q, k, v, c.tree)))
    for a, b in zip(*got):
        assert_same_bits(a, b, "wide strides")
    near = torch.stack([c.k, c.v])[None].contiguous()
    for a, b in zip(kinv.tree_accept(c.tree, tok_, nxt, near), kinv.tree_accept(c.tree, tok_, nxt, kv)):
        assert torch.equal(a, b)
    assert_same_bits(kv, near, "the moved slots")
    assert kinv.last_device_status() == 0


def test_captured_accept_follows_its_tensors(kinv):
    parents, n = shape_parents("bushy", 40, 5), 40
    t = [torch.tensor(x, **I32) for x in ([7], [n], [0], parents)]
    tree = kinv.Tree(*t, 64, 80)
    tok, nxt = torch.zeros(n, **I32), torch.zeros(n, **I32)
    kv = synth.normal_bf16((2, 2, 1, 80, 2, 64), 1.0, 4, "cuda")
    start = kv.clone()
    outs = [torch.empty(1, **I32), torch.empty(1, 64, **I32), torch.empty(1, 64, **I32)]
    call = lambda: kinv.tree_accept(tree, tok, nxt, kv, *outs)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed, ctx in ((1, 7), (2, 0), (3, 40)):
        t[0].fill_(ctx)
        tok.copy_(synth.uniform_int(n, 0, 2, seed)), nxt.copy_(synth.uniform_int(n, 0, 2, seed + 9))
        kv.copy_(start)
        g.replay()
        want = otree.accept(parents, tok.tolist(), nxt.tolist())
        assert outs[0].tolist() == [len(want)] and outs[1][0, : len(want)].tolist() == want
        for i, j in enumerate(want):
            assert_same_bits(kv[:, :, 0, ctx + i], start[:, :, 0, ctx + j], f"slot {i}")


@pytest.mark.parametrize("hq,hkv,d,n,B,slots", [(32, 8, 128, 4, 18, 1100), (8, 1, 128, 1, 130, 1100), (32, 8, 128, 9, 14, 1100), (32, 8, 128, 5, 66, 1100), (8, 1, 64, 3, 180, 1800),
                                                (2, 2, 64, 33, 33, 2100)])
def test_small_trees_of_many_sequences(kinv, hq, hkv, d, n, B, slots):
    """Trees of 8 to 36 (node, head) pairs in batches that take the tensor-core
    path: groups of 16 pairs that are not full, ragged down to one node."""
    ctx = [(37 * b * b + 5) % (slots - n) for b in range(B)]
    parents = [shape_parents(["bushy", "chain", "forest"][b % 3], 1 + (b * 7) % n if b else n, b) for b in range(B)]
    c = Case(kinv, ctx, parents, hq, hkv, d, slots=slots, seed=130)
    out = c.run()
    assert kinv.last_device_status() == 0
    c.check_bits(out, "small trees")


@pytest.mark.parametrize("B,n,ctx", [(1, 64, 8000), (4, 16, 4000), (8, 4, 6000), (1, 64, 700)])
def test_steps_behind_each_other(kinv, B, n, ctx):
    """Rotation and attention of changing rows with nothing waiting in between: the
    kernels of a step start early, but not before the rows are there.  On two streams
    at once, then in one graph."""
    def setup(seed):
        c = Case(kinv, [ctx - 37 * b for b in range(B)], [shape_parents("bushy", n, b) for b in range(B)], 32, 8, 128,
                 seed=seed, poison=False)
        qkv = [synth.normal_bf16((c.rows, 48 * 128), 1.0, seed + 9 + i, "cuda") for i in range(3)]
        ws = torch.empty(kinv.attn_tree_workspace(c.tree, 32, 8, 128), dtype=torch.uint8, device="cuda")
        q = torch.empty(c.rows, 32, 128, dtype=torch.bfloat16, device="cuda")

        def step(i, out):
            kinv.rope_append_tree(qkv[i % 3], q, c.k, c.v, c.tree, 32, 8, 128, 1e6)
            return kinv.attn_tree(q, c.k, c.v, c.tree, out=out, workspace=ws)

        want = []
        for i in range(3):
            want.append(step(i, torch.empty_like(q)))
            torch.cuda.synchronize()
        return step, want

    sides = [setup(200), setup(300)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for i in range(60):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                outs[k].append(sides[k][0](i, torch.empty_like(sides[k][1][0])))
    torch.cuda.synchronize()
    for k in (0, 1):
        for i, o in enumerate(outs[k]):
            assert_same_bits(o, sides[k][1][i % 3], f"side {k} step {i}")
    step, want = sides[0]
    outs = [torch.empty_like(want[0]) for _ in range(7)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i, o in enumerate(outs):
            step(i, o)
    for _ in range(5):
        for o in outs:
            o.zero_()
        g.replay()
        for i, o in enumerate(outs):
            assert_same_bits(o, want[i % 3], f"captured step {i}")
    assert kinv.last_device_status() == 0
