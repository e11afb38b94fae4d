"""Arguments of the drafted-tree calls that no kernel may be given (no GPU: the
tensors and the library are stand-ins)."""
import pytest

from invariant_deterministic_gb300 import kinv
from test_stream_memory_host import BF, F32, U8, Tensor, tree, world  # noqa: F401


def host(t):
    t.is_cuda = False
    return t


@pytest.mark.parametrize("workspace", [host(Tensor((8192,), U8)), host(Tensor((1 << 20,), F32))])
def test_attn_tree_refuses_scratch_in_host_memory(world, workspace):  # noqa: F811
    q, k = Tensor((10, 4, 64), BF), Tensor((2, 512, 2, 64), BF)
    with pytest.raises(ValueError):
        kinv.attn_tree(q, k, k, tree(), workspace=workspace)
    assert not world.calls
    kinv.attn_tree(q, k, k, tree(), workspace=Tensor((8192,), U8))
    assert len(world.calls) == 1
