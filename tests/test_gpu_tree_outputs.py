"""What drafted-tree calls return for sequences that they leave out."""
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth
from test_gpu_tree import Case, shape_parents

pytestmark = gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


@pytest.mark.parametrize("broken", [(1, 400, 0), (1, 99, 1), (1, -1, 2), ("parent", 3, 3)])
def test_acceptance_of_a_broken_tree_is_empty(kinv, broken):
    parents = [shape_parents("bushy", 9, 1), shape_parents("chain", 6), shape_parents("star", 5)]
    c = Case(kinv, [100, 300, 20], parents, 4, 2, 64, seed=500, slots=310)
    tok = torch.zeros(c.rows, **I32)
    want = [t.clone() for t in kinv.tree_accept(c.tree, tok, tok)]
    index, value, which = broken
    t = [x.clone() for x in c.tree.tensors]
    t[which][c.off[1] + 3 if index == "parent" else index] = value
    tree = kinv.Tree(*t, c.tree.max_nodes, c.tree.max_kv)
    for _ in range(3):      # memory that held plausible values of another call
        left = [torch.full((n,), 3, **I32) for n in (3, 3, 27, 27, 54, 54) for _ in range(4)]
        del left
        got = kinv.tree_accept(tree, tok, tok)
        assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
        assert got[0].tolist() == [want[0][0].item(), 0, want[0][2].item()]
        for a, b in zip(got[1:], want[1:]):
            assert torch.all(a[1] == -1)
            assert_same_bits(a[::2], b[::2], "beside it")
        # given outputs keep what they held; any one of them alone
        held = torch.full((3,), -5, **I32), torch.full((3, 9), -6, **I32), torch.full((3, 9), -7, **I32)
        for k, name in enumerate(("n_accepted", "path", "out_tokens")):
            mine = held[k].clone()
            mixed = kinv.tree_accept(tree, tok, tok, **{name: mine})
            assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
            assert mixed[k] is mine and torch.all(mine[1] == held[k][1])
            for i, t in enumerate(mixed):
                if i != k:
                    assert_same_bits(t, got[i], "the others")
