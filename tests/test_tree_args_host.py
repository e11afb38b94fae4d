"""Arguments of the drafted-tree calls that no kernel may be given (no GPU: the
tensors and the library are stand-ins)."""
import pytest

from invariant_deterministic_gb300 import kinv
from test_stream_memory_host import BF, F32, U8, Tensor, tree, world  # noqa: F401


def host(t):
    t.is_cuda = False
    return t


def strided(t):
    t.is_contiguous = lambda: False
    return t


@pytest.mark.parametrize("workspace", [host(Tensor((8192,), U8)), host(Tensor((1 << 20,), F32))])
def test_attn_tree_refuses_scratch_in_host_memory(world, workspace):  # noqa: F811
    q, k = Tensor((10, 4, 64), BF), Tensor((2, 512, 2, 64), BF)
    with pytest.raises(ValueError):
        kinv.attn_tree(q, k, k, tree(), workspace=workspace)
    assert not world.calls
    kinv.attn_tree(q, k, k, tree(), workspace=Tensor((8192,), U8))
    assert len(world.calls) == 1


@pytest.mark.parametrize("gain,error", [
    (Tensor((64,), F32), TypeError),            # read as bf16: every other value the low half of a float
    (host(Tensor((64,), BF)), ValueError),
    (Tensor((32,), BF), ValueError),            # half a head
    (strided(Tensor((64,), BF)), ValueError),
])
@pytest.mark.parametrize("which", ["q_norm", "k_norm"])
def test_rope_append_tree_refuses_gains(world, which, gain, error):  # noqa: F811
    k = Tensor((2, 512, 2, 64), BF)
    call = lambda **g: kinv.rope_append_tree(Tensor((10, 512), BF), Tensor((10, 4, 64), BF), k, k, tree(), 4, 2, 64, 1e4, **g)
    with pytest.raises(error):
        call(**{which: gain})
    assert not world.calls
    call(**{which: Tensor((64,), BF)})
    call()
    assert len(world.calls) == 2
