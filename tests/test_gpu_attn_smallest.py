"""Attention over a cache of no slots: zeros, and any other length reported."""
import pytest
import torch

from helpers import ensure_lib, gpu

pytestmark = gpu

NEVER_READ = 0x10000


@pytest.fixture(scope="module")
def kinv():
    return ensure_lib()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 2)])
@pytest.mark.parametrize("lens,status", [([0, 0, 0], "OK"), ([0, 1, 0], "ERR_INVALID_ARG"), ([0, 0, -1], "ERR_INVALID_ARG")])
@pytest.mark.parametrize("call", ["decode8 e4m3", "decode8 int8", "decode_window"])
def test_a_cache_of_no_slots_gives_zeros(kinv, call, d, window, sinks, lens, status):
    hq, hkv, bsz = 4, 2, len(lens)
    L = kinv.lib()
    q = torch.ones(bsz, hq, d, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    if call == "decode_window":
        assert L.kinv_attn_decode_window_workspace(bsz, hq, d, 0, 256, window, sinks) == 0
        st = L.kinv_attn_decode_window(q.data_ptr(), NEVER_READ, NEVER_READ, hkv * d, hkv * d, n.data_ptr(), out.data_ptr(), bsz, hq, hkv, d, 0,
                                       256, window, sinks, 0.0, None, 0, stream)
    else:
        c = kinv.Cache8Struct(k=NEVER_READ, v=NEVER_READ, k_exp=NEVER_READ, v_exp=NEVER_READ, seq_stride=hkv * d, tok_stride=hkv * d,
                              exp_seq_stride=hkv, exp_head_stride=1, B=bsz, slots=0, dtype=kinv.I8 if "int8" in call else kinv.E4M3)
        assert L.kinv_attn_decode8_workspace(bsz, hq, d, 0, window, sinks, 256) == 0
        st = L.kinv_attn_decode8(q.data_ptr(), kinv.ctypes.byref(c), n.data_ptr(), out.data_ptr(), bsz, hq, hkv, d, 256, window, sinks, 0.0,
                                 None, 0, stream)
    assert st == kinv.OK
    assert kinv.last_device_status() == getattr(kinv, status)
    assert (out == 0).all()
