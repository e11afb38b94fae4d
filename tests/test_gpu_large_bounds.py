"""Host-side bounds far above what the call holds (2^31 - 1 says "whatever it is"): the
same results, and lengths that do not fit still reported."""
import pytest
import torch

from helpers import assert_same_bits, ensure_lib, gpu, synth

pytestmark = gpu

I32 = dict(dtype=torch.int32, device="cuda")
MOST = 2**31 - 1


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


def i32(v):
    return torch.tensor(v, **I32)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (2, 2, 64)])
@pytest.mark.parametrize("most", [1 << 20, MOST - 20, MOST])
def test_prefill_with_a_large_bound_of_rows(kinv, hq, hkv, d, most):
    start, n, off = [700, 0, 300], [40, 0, 200], [0, 40, 40]
    k, v = (synth.normal_bf16((3, 900, hkv, d), 1.0, s, "cuda") for s in (1, 2))
    q = synth.normal_bf16((240, hq, d), 1.0, 3, "cuda")
    args = (i32(start), i32(n), i32(off))
    ref = kinv.attn_prefill(q, k, v, *args, 200, 900, window=250, sinks=2)
    assert_same_bits(kinv.attn_prefill(q, k, v, *args, most, 900, window=250, sinks=2), ref, "bf16")
    c = kinv.Cache8.empty(3, 900, hkv, d, "int8")
    kinv.cache8_write(c, k, v, i32([0] * 3), i32([900] * 3))
    ref = kinv.attn_prefill8(q, c, *args, 200, 900)
    ws = torch.empty(kinv.attn_prefill8_workspace(3, 240, hq, hkv, d, 900), dtype=torch.uint8, device="cuda")
    if (most + 128 * hkv // hq - 1) // (128 * hkv // hq) * hkv * 3 <= 0x7F000000:   # tiles of the bound
        assert_same_bits(kinv.attn_prefill8(q, c, *args, most, 900, workspace=ws), ref, "int8")
    assert kinv.last_device_status() == 0
    for bad in ((i32([700, 0, 300]), i32([40, 0, 241]), i32([0, 40, 0])), (i32([700, 0, 300]), i32([40, 0, 601]), i32([0, 40, 40]))):
        out = torch.full_like(q, 7.0)
        kinv.attn_prefill(q, k, v, *bad, most, 900, out=out, window=250, sinks=2)
        assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
        assert (out[40:] == 7).all() and (out[:40] != 7).any()


@pytest.mark.parametrize("most", [65, MOST - 20, MOST])
def test_write_and_read_with_a_large_bound_of_tokens(kinv, most):
    hkv, d, slots = 2, 64, 64
    k, v = (synth.normal_bf16((2, slots, hkv, d), 1.0, s, "cuda") for s in (1, 2))
    start, n = i32([0, 10]), i32([64, 50])
    L, stream = kinv.lib(), torch.cuda.current_stream().cuda_stream
    ref, c = kinv.Cache8.empty(2, slots, hkv, d), kinv.Cache8.empty(2, slots, hkv, d)
    kinv.cache8_write(ref, k, v, start, n)
    strides = (slots * hkv * d, hkv * d)
    assert L.kinv_cache8_write(k.data_ptr(), v.data_ptr(), *strides, c.ptr, start.data_ptr(), n.data_ptr(), 2, most, hkv, d, stream) == kinv.OK
    for a, b in zip(c.tensors, ref.tensors):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    want = kinv.cache8_read(ref, start, n, k=torch.zeros_like(k), v=torch.zeros_like(v))
    got = torch.zeros_like(k), torch.zeros_like(v)
    assert L.kinv_cache8_read(c.ptr, start.data_ptr(), n.data_ptr(), got[0].data_ptr(), got[1].data_ptr(), *strides, 2, most, hkv, d,
                              stream) == kinv.OK
    for a, b in zip(got, want):
        assert_same_bits(a, b, "read back")
    assert kinv.last_device_status() == 0
    n[1] = 65                                 # more than there are slots: left out, reported
    before = [t.clone() for t in c.tensors]
    assert L.kinv_cache8_write(k.data_ptr(), v.data_ptr(), *strides, c.ptr, start.data_ptr(), n.data_ptr(), 2, most, hkv, d, stream) == kinv.OK
    assert kinv.last_device_status() == kinv.ERR_INVALID_ARG
    for a, b in zip(c.tensors, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
