"""Every way a call of kinv_attn_tree may be split into launches, against the
decode step's bits, and rows that meet infinities and NaN on each of them.

Which kernels a call takes follows from the bounds of its tree (B, max_nodes,
max_kv) and its heads alone; G = Hq / Hkv, pairs = max_nodes G, triples =
B Hkv floor(max_kv / 256), S = ceil(max_kv / 256):
  tensor cores for the context: triples pairs >= 5120 beyond 16 pairs, else
    D = 128 and triples >= 512;
  one cluster launch: not the above, S <= 8, few tiles of 16 pairs;
  else the split kernel alone takes the context, in tiles of 16 or of 32 pairs."""
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth
from test_gpu_tree import Case, shape_parents

pytestmark = gpu


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def assert_same_values(a, b, what):
    """Bit equality where the values are numbers, NaN against NaN (of any sign) elsewhere."""
    na, nb = torch.isnan(a), torch.isnan(b)
    assert torch.equal(na, nb), f"{what}: NaN in other places"
    assert_same_bits(torch.where(na, torch.zeros_like(a), a), torch.where(nb, torch.zeros_like(b), b), what)


SPLIT = [  # hq, hkv, d, nodes, contexts: the split kernel for every split
    (32, 8, 128, 4, [7990]),                          # one tile of 16 pairs, 32 splits
    (32, 8, 128, 3, [2100, 5000, 0, 255]),            # ragged, without whole splits in between
    (8, 1, 64, 2, [9000, 1, 4096]),                   # D = 64 with at most 16 pairs, at any length
    (2, 2, 128, 16, [6000]),                          # a node per pair
    (32, 8, 128, 40, [300, 256]),                     # tiles of 32 pairs
    (4, 2, 64, 64, [436, 255, 256, 257, 0, 300, 17, 400, 31, 288]),
    (2, 2, 64, 64, [336 - 17 * i for i in range(19)]),
    (32, 8, 128, 64, [700]),                          # sixteen tiles of 16 pairs
    (8, 1, 128, 64, [1500]),                          # 512 pairs, more than one group of 128
]


@pytest.mark.parametrize("hq,hkv,d,n,ctx", SPLIT, ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}x")
@pytest.mark.parametrize("shape", ["bushy", "chain", "forest"])
def test_the_split_kernel_alone(kinv, hq, hkv, d, n, ctx, shape):
    parents = [shape_parents(shape, n if b == 0 else 1 + (5 * b) % n, b) for b in range(len(ctx))]
    c = Case(kinv, ctx, parents, hq, hkv, d, seed=300, gap=1)
    out = torch.full_like(c.q, 7.0)
    c.run(out=out)
    assert kinv.last_device_status() == 0
    c.check_bits(out, shape)


@pytest.mark.parametrize("hq,hkv,d,n,ctx,slots", [
    (4, 2, 64, 13, [1021, 1000, 0, 255, 513, 900, 256], 1060),    # five blocks a cluster
    (32, 8, 128, 4, [1290, 40], 1300), (32, 8, 128, 4, [1536, 1023], 1700), (32, 8, 128, 4, [2036, 1792], 2040),
    (8, 1, 64, 2, [2030, 0, 1600], 2048), (2, 2, 128, 16, [1700, 1279], 1716), (8, 1, 128, 6, [1400], 1406)])
@pytest.mark.parametrize("shape", ["bushy", "chain"])
def test_clusters_of_five_to_eight(kinv, hq, hkv, d, n, ctx, slots, shape):
    parents = [shape_parents(shape, n - b % n, b) for b in range(len(ctx))]
    c = Case(kinv, ctx, parents, hq, hkv, d, slots=slots, seed=310)
    out = c.run()
    assert kinv.last_device_status() == 0
    c.check_bits(out, shape)


PATHS = {  # hq, hkv, d, nodes, contexts, slots
    "tensor cores, one tile": (32, 8, 128, 20, [4000, 700], 4100),
    "tensor cores, two tiles": (32, 8, 128, 48, [3000, 1100], 3100),
    "tensor cores, 16 pairs": (32, 8, 128, 4, [9000, 9100], 9200),
    "tensor cores, D = 64": (8, 1, 64, 16, [9000, 5000], 9100),
    "one cluster": (32, 8, 128, 4, [1500, 600], 1600),
    "split kernel": (32, 8, 128, 4, [5000, 600], 5100),
}


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("where", ["k", "v"])
def test_rows_that_meet_infinities(kinv, path, value, where):
    """A value that is no number, or the type's lowest, in the first split, in a later
    one and at a drafted node: the rows that see it have decode's values, those of the
    other sequence and of nodes off its path the bits they have without it."""
    hq, hkv, d, n, ctx, slots = PATHS[path]
    parents = [shape_parents("bushy", n, 1), shape_parents("chain", min(n, 5))]
    c = Case(kinv, ctx, parents, hq, hkv, d, slots=slots, seed=320)
    clean = c.run()
    c.check_bits(clean, path)
    t = c.k if where == "k" else c.v
    last = n - 1
    for slot in (3, 515, ctx[0] - 1, ctx[0] + last):
        keep = t[0, slot].clone()
        t[0, slot] = value
        out = c.run()
        assert_same_values(out[: n], c.decode(0), f"slot {slot}")
        assert_same_bits(out[c.off[1]:], clean[c.off[1]:], f"the other sequence, slot {slot}")
        if slot == ctx[0] + last:   # the last node is nobody's ancestor
            assert_same_bits(out[:last], clean[:last], "nodes off its path")
        t[0, slot] = keep
    assert kinv.last_device_status() == 0


def test_a_whole_split_of_masks(kinv):
    """Splits whose scores are all -infinity, and the tensor-core fold behind them."""
    c = Case(kinv, [2000, 900], [shape_parents("bushy", 20, 1), shape_parents("chain", 6)], 32, 8, 128, slots=4100, seed=330)
    c.q.abs_()
    for lo in (0, 256, 1024):
        keep = c.k[0, lo: lo + 256].clone()
        c.k[0, lo: lo + 256] = float("-inf")
        assert_same_values(c.run()[:20], c.decode(0), f"split at {lo}")
        c.k[0, lo: lo + 256] = keep
    c.check_bits(c.run(), "without them")


@pytest.mark.parametrize("path", PATHS)
def test_calls_repeat_their_bits(kinv, path):
    hq, hkv, d, n, ctx, slots = PATHS[path]
    c = Case(kinv, ctx, [shape_parents("bushy", n, 1), shape_parents("chain", min(n, 5))], hq, hkv, d, slots=slots, seed=340)
    want = c.run()
    ws = torch.empty(kinv.attn_tree_workspace(c.tree, hq, hkv, d), dtype=torch.uint8, device="cuda")
    for i in range(20):
        ws.fill_(0xFF if i % 2 else 0)
        assert_same_bits(c.run(workspace=ws), want, f"call {i}")
    c.check_bits(want, path)
