"""Thin ctypes binding over libkinv.so (the C ABI in ``include/kinv.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  Tensors are PyTorch CUDA tensors (PyTorch supplies
device memory and the current stream); each wrapper checks dtypes and
contiguity, passes raw pointers, sizes and the current stream, and raises
``KinvError`` if the library returns a non-zero status.  There is no fallback:
if the library has not been built, loading it raises.

``stream=`` names the stream a call is enqueued on (default: the current one).
The call waits for nothing on other streams: its inputs have to be ready there,
and whoever reads its results elsewhere waits for it.  What a call allocates is
that stream's memory.  The calls on drafted trees, logprobs, the 8-bit cache and
windowed attention hold their inputs' memory for it too; for the others the caller
keeps the inputs until they are done.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from functools import partial

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkinv.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = (
    0, -1, -2, -3, -4, -5, -6)
BF16, F32, E4M3, I8 = 0, 1, 2, 3
SPLIT_LEN = 256

_lib = None

_c_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int
_f32 = ctypes.c_float
_sz = ctypes.c_size_t

# name -> (restype, argtypes); mirrors include/kinv.h
SIGNATURES = {
    "kinv_status_string": (ctypes.c_char_p, [_i32]),
    "kinv_device_class": (ctypes.c_char_p, []),
    "kinv_build_id": (ctypes.c_char_p, []),
    "kinv_last_device_status": (_i32, [_c_p]),
    "kinv_test_bounded_wait": (_i32, [_i64, _c_p]),
    "kinv_gemm": (_i32, [_c_p, _i64, _c_p, _i64, _c_p, _i64, _i32, _i32, _i32, _i32, _c_p]),
    "kinv_gemm_fused": (_i32, [_c_p, _i64, _c_p, _i64, _c_p, _i64, _i32, _i32, _i32, _i32, _c_p, _c_p]),
    "kinv_row_sumsq": (_i32, [_c_p, _i64, _i32, _i32, _c_p, _c_p]),
    "kinv_gemm_swiglu": (_i32, [_c_p, _i64, _c_p, _i64, _c_p, _i64, _i32, _i32, _i32, _c_p, _c_p]),
    "kinv_gemm_qkv_rope": (_i32, [_c_p, _i64, _c_p, _i64, _c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p,
                                  _c_p, _c_p, _f32, _i32, _i32, _i32, _i32, _i32, _f32, _c_p, _c_p]),
    "kinv_rmsnorm": (_i32, [_c_p, _i64, _c_p, _c_p, _c_p, _i64, _i32, _i32, _f32, _c_p]),
    "kinv_attn_decode_workspace": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "kinv_attn_decode": (_i32, [_c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _i32, _i32, _i32, _i32,
                                _i32, _i32, _f32, _c_p, _sz, _c_p]),
    "kinv_attn_decode_noalloc": (_i32, [_c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _i32, _i32, _i32,
                                        _i32, _i32, _i32, _f32, _c_p]),
    "kinv_attn_prefill_workspace": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "kinv_attn_prefill": (_i32, [_c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _c_p, _c_p, _i32, _i32,
                                 _i32, _i32, _i32, _i32, _i32, _i32, _f32, _c_p, _sz, _c_p]),
    "kinv_attn_decode_window_workspace": (_sz, [_i32] * 7),
    "kinv_attn_decode_window": (_i32, [_c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _i32, _i32, _i32, _i32, _i32,
                                       _i32, _i32, _i32, _f32, _c_p, _sz, _c_p]),
    "kinv_attn_prefill_window": (_i32, [_c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _c_p, _c_p, _i32, _i32, _i32,
                                        _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _c_p, _sz, _c_p]),
    "kinv_attn_prefill_window_workspace": (_sz, [_i32] * 9),
    "kinv_rope_append8": (_i32, [_c_p, _i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _f32, _i32, _i32, _i32, _i32,
                                 _f32, _c_p]),
    "kinv_cache8_write": (_i32, [_c_p, _c_p, _i64, _i64, _c_p, _c_p, _c_p, _i32, _i32, _i32, _i32, _c_p]),
    "kinv_cache8_read": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _i32, _i32, _i32, _i32, _c_p]),
    "kinv_attn_decode8_workspace": (_sz, [_i32] * 7),
    "kinv_attn_decode8": (_i32, [_c_p, _c_p, _c_p, _c_p, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _c_p,
                                 _sz, _c_p]),
    "kinv_attn_prefill8_workspace": (_sz, [_i32] * 7),
    "kinv_attn_prefill8": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                  _i32, _i32, _i32, _f32, _c_p, _sz, _c_p]),
    "kinv_sample_workspace": (_sz, [_i32, _i32]),
    "kinv_sample": (_i32, [_c_p, _i64, _i32, _i32, _c_p, _c_p, _i32, _c_p, _c_p, _c_p, _c_p, _sz,
                           _c_p]),
    "kinv_embed": (_i32, [_c_p, _i32, _i32, _c_p, _c_p, _i32, _c_p]),
    "kinv_add": (_i32, [_c_p, _c_p, _c_p, _i64, _c_p]),
    "kinv_scale_columns": (_i32, [_c_p, _i64, _c_p, _c_p, _i64, _i32, _i32, _c_p]),
    "kinv_swiglu": (_i32, [_c_p, _i64, _c_p, _i64, _i32, _i32, _c_p]),
    "kinv_rope_append": (_i32, [_c_p, _i64, _c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _c_p, _c_p,
                                _f32, _i32, _i32, _i32, _i32, _f32, _c_p]),
    "kinv_rope_append_tree": (_i32, [_c_p, _i64, _c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _c_p, _f32,
                                     _i32, _i32, _i32, _f32, _c_p]),
    "kinv_attn_tree_workspace": (_sz, [_i32] * 8),
    "kinv_attn_tree": (_i32, [_c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _i32, _i32, _i32, _i32, _f32,
                              _c_p, _sz, _c_p]),
    "kinv_tree_accept": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i32, _i64, _i64, _i64, _i32, _i32, _c_p,
                                _c_p, _c_p, _c_p]),
    "kinv_tree_accept_marked": (_i32, [_c_p, _c_p, _c_p, _c_p, _c_p, _i32, _i64, _i64, _i64, _i32, _i32, _c_p,
                                       _c_p, _c_p, _i32, _c_p]),
    "kinv_logprobs": (_i32, [_c_p, _i32, _i64, _i32, _i32, _c_p, _i32, _c_p, _c_p, _i32, _c_p, _c_p, _c_p]),
    "kinv_decode_advance": (_i32, [_c_p, _c_p, _i32, _c_p, _c_p, _c_p, _c_p, _i32, _c_p]),
}


class KinvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """Load libkinv.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libkinv.so is not built ({LIB_PATH}); run "
                               "invariant_deterministic_gb300.build.build() first")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def status_string(status: int) -> str:
    return lib().kinv_status_string(int(status)).decode()


def device_class() -> str:
    return lib().kinv_device_class().decode()


def build_id() -> str:
    return lib().kinv_build_id().decode()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise KinvError(status, where)


# the current stream's handle without building a Stream object (0.1 against 3
# microseconds a call), where this PyTorch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_INT_MAX = 2**31 - 1


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _get_device is not None:
        return _raw_stream(_get_device())
    return torch.cuda.current_stream().cuda_stream


def _side(stream):
    """``stream`` where it is another than the current one, else None."""
    return None if stream is None or stream.cuda_stream == _stream() else stream


def _scratch(side, make, *args, **kw):
    """make(...), of the memory of the stream that the call runs on: a block of
    the current stream's may be handed out again, or still be in use there,
    while a kernel on another stream writes it."""
    if side is None:
        return make(*args, **kw)
    with torch.cuda.stream(side):
        return make(*args, **kw)


def _output(side, make, *args, **kw):
    """The same for a tensor that goes to the caller, who reads it on the current
    stream and may drop it there."""
    t = _scratch(side, make, *args, **kw)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _empty(side):
    """torch.empty for what a call returns."""
    return torch.empty if side is None else partial(_output, side, torch.empty)


def _empty_like(side):
    return torch.empty_like if side is None else partial(_output, side, torch.empty_like)


def _hold(side, *tensors) -> None:
    """The memory of these is not reused before the call on ``side`` is done with
    it, even if the caller drops them."""
    for t in tensors:
        if t is not None:
            t.record_stream(side)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")


def last_device_status(stream=None) -> int:
    return lib().kinv_last_device_status(_stream(stream))


def test_bounded_wait(limit_ns: int, stream=None) -> None:
    """kinv_test_bounded_wait: one block waits on a barrier nothing
    completes, gives up after limit_ns and records KINV_ERR_TIMEOUT."""
    _check(lib().kinv_test_bounded_wait(int(limit_ns), _stream(stream)), "kinv_test_bounded_wait")


# --------------------------------------------------------------------- GEMM
def gemm(a: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None,
         out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """out[M][N] = a[M][K] . w[N][K]^T (bf16 in, fp32 accumulate)."""
    _need(a, torch.bfloat16, "a")
    _need(w, torch.bfloat16, "w")
    m, k = a.shape
    n = w.shape[0]
    if w.shape[1] != k or a.stride(1) != 1 or w.stride(1) != 1:
        raise ValueError("gemm: shapes or layouts do not match")
    if out is None:
        out = _empty(_side(stream))(m, n, dtype=out_dtype, device=a.device)
    if out.stride(1) != 1 or tuple(out.shape) != (m, n):
        raise ValueError("gemm: bad output")
    dt = F32 if out.dtype == torch.float32 else BF16
    _check(lib().kinv_gemm(_ptr(a), a.stride(0), _ptr(w), w.stride(0), _ptr(out), out.stride(0),
                           dt, m, n, k, _stream(stream)), "kinv_gemm")
    return out


class GemmFusion(ctypes.Structure):
    """kinv_gemm_fusion: the RMSNorm folded into the projections around it."""
    _fields_ = [("row_ss", _c_p), ("row_ss_tiles", _i32), ("norm_dim", _i32), ("eps", _f32),
                ("resid", _c_p), ("ld_resid", _i64), ("ss_out", _c_p)]


def norm_in(row_ss: torch.Tensor, norm_dim: int, eps: float) -> GemmFusion:
    """Consuming side: scale output row m by 1/rms from row_ss [M][tiles]."""
    _need(row_ss, torch.float32, "row_ss")
    return GemmFusion(row_ss=_ptr(row_ss), row_ss_tiles=row_ss.shape[1], norm_dim=norm_dim, eps=float(eps))


def residual_out(resid: torch.Tensor, ss_out: torch.Tensor) -> GemmFusion:
    """Producing side: resid <- bf16(resid + out), out the fp32 product
    (rounded once); ss_out [M][N/128]."""
    _need(resid, torch.bfloat16, "resid")
    _need(ss_out, torch.float32, "ss_out")
    return GemmFusion(resid=_ptr(resid), ld_resid=resid.stride(0), ss_out=_ptr(ss_out))


def _fusion_ptr(f):
    return ctypes.byref(f) if f is not None else None


def gemm_fused(a, w, fusion: GemmFusion, out=None, n=None, stream=None):
    """kinv_gemm_fused.  With a residual fusion there is no other output
    (out may be None); otherwise out is written as by gemm()."""
    _need(a, torch.bfloat16, "a")
    _need(w, torch.bfloat16, "w")
    m, k = a.shape
    n = w.shape[0] if n is None else n
    dt = F32 if (out is not None and out.dtype == torch.float32) else BF16
    _check(lib().kinv_gemm_fused(_ptr(a), a.stride(0), _ptr(w), w.stride(0), _ptr(out),
                                 out.stride(0) if out is not None else n, dt, m, n, k,
                                 _fusion_ptr(fusion), _stream(stream)), "kinv_gemm_fused")
    return out


def row_sumsq(x, ss_out, stream=None):
    """ss_out[r][t] = sum of x[r][128t .. 128t+127]^2 (fp32)."""
    _need(x, torch.bfloat16, "x")
    _need(ss_out, torch.float32, "ss_out")
    rows, dim = x.shape
    _check(lib().kinv_row_sumsq(_ptr(x), x.stride(0), rows, dim, _ptr(ss_out), _stream(stream)),
           "kinv_row_sumsq")
    return ss_out


def interleave_gate_up(w_gu: torch.Tensor) -> torch.Tensor:
    """[gate rows; up rows] ([2F][K]) -> the block-of-64 interleaved layout
    kinv_gemm_swiglu reads (a one-time weight layout change, a copy)."""
    two_f, k = w_gu.shape
    f = two_f // 2
    return w_gu.view(2, f // 64, 64, k).permute(1, 0, 2, 3).reshape(two_f, k).contiguous()


def gemm_swiglu(a: torch.Tensor, w_gu_il: torch.Tensor, out: torch.Tensor | None = None,
                fusion: GemmFusion | None = None, stream=None) -> torch.Tensor:
    """act[M][F] = bf16(silu(a . Wgate^T) * (a . Wup^T)), W in the interleaved
    layout of ``interleave_gate_up``."""
    _need(a, torch.bfloat16, "a")
    _need(w_gu_il, torch.bfloat16, "w_gu")
    m, k = a.shape
    f = w_gu_il.shape[0] // 2
    if out is None:
        out = _empty(_side(stream))(m, f, dtype=torch.bfloat16, device=a.device)
    _check(lib().kinv_gemm_swiglu(_ptr(a), a.stride(0), _ptr(w_gu_il), w_gu_il.stride(0), _ptr(out),
                                  out.stride(0), m, f, k, _fusion_ptr(fusion), _stream(stream)),
           "kinv_gemm_swiglu")
    return out


def gemm_qkv_rope(a, w_qkv, q_out, k_cache, v_cache, seq, pos, n_q, n_kv, head_dim, rope_base,
                  q_norm=None, k_norm=None, eps=1e-6, fusion=None, stream=None):
    """kinv_gemm followed by kinv_rope_append in one kernel: q heads of
    a . w_qkv^T -> q_out [M][Hq][D]; k and v heads into the caches
    [B][Lmax][Hkv][D] at [seq][pos]."""
    _need(a, torch.bfloat16, "a")
    _need(w_qkv, torch.bfloat16, "w_qkv")
    m, k = a.shape
    _check(lib().kinv_gemm_qkv_rope(_ptr(a), a.stride(0), _ptr(w_qkv), w_qkv.stride(0), _ptr(q_out),
                                    _ptr(k_cache), _ptr(v_cache), k_cache.stride(0), k_cache.stride(1),
                                    _ptr(seq), _ptr(pos), _ptr(q_norm), _ptr(k_norm),
                                    float(eps), m, n_q, n_kv, head_dim, k, float(rope_base),
                                    _fusion_ptr(fusion), _stream(stream)),
           "kinv_gemm_qkv_rope")
    return q_out


# ------------------------------------------------------------------ RMSNorm
def rmsnorm(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, residual=None, out=None,
            stream=None) -> torch.Tensor:
    """y = RMSNorm(x) * w; with ``residual``, x <- bf16(x + residual) first
    (in place) and y = RMSNorm(x)."""
    _need(x, torch.bfloat16, "x")
    rows, dim = x.shape
    if out is None:
        out = _empty_like(_side(stream))(x)
    _check(lib().kinv_rmsnorm(_ptr(x), x.stride(0), _ptr(residual), _ptr(w), _ptr(out),
                              out.stride(0), rows, dim, float(eps), _stream(stream)),
           "kinv_rmsnorm")
    return out


# ---------------------------------------------------------------- attention
def attn_decode_workspace(batch: int, n_q: int, head_dim: int, max_len: int,
                          split_len: int = SPLIT_LEN, window: int = 0, sinks: int = 0) -> int:
    if window:
        return int(lib().kinv_attn_decode_window_workspace(batch, n_q, head_dim, max_len, split_len, window, sinks))
    return int(lib().kinv_attn_decode_workspace(batch, n_q, head_dim, max_len, split_len))


def _here(*named) -> None:
    """The tensors lie on the current device, whose stream a call runs on."""
    dev = 0 if _get_device is None else _get_device()
    for name, t in named:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name}: expected a tensor on the current CUDA device, got one on {t.device}")


def _window_ints(window: int, sinks: int) -> None:
    if window > _INT_MAX or sinks > _INT_MAX:
        raise ValueError("window and sinks are 32-bit numbers")


def _rows_of(q, out, what: str) -> None:
    """q and out [rows][Hq][D], bf16 and contiguous."""
    bf = torch.bfloat16
    if not (q.dtype is bf and q.is_contiguous() and q.dim() == 3
            and (out is None or (out.dtype is bf and out.is_contiguous() and out.shape == q.shape))):
        _need(q, bf, "q")
        if out is not None:
            _need(out, bf, "out")
        raise ValueError(f"{what}: q and out must be contiguous [rows][Hq][D] of one shape")


def _window_caches(k_cache, v_cache, batch: int, head_dim: int, what: str):
    """Checks of the windowed calls' caches: (shape, strides)."""
    bf = torch.bfloat16
    if not k_cache.dtype is v_cache.dtype is bf:
        _need(k_cache, bf, "k_cache")
        _need(v_cache, bf, "v_cache")
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or v_cache.stride() != stride:
        raise ValueError(f"{what}: the caches must be [B][slots][Hkv][D] and share shape and strides")
    if stride[3] != 1 or (stride[2] != head_dim and shape[2] > 1) or shape[3] != head_dim or shape[0] < batch:
        raise ValueError(f"{what}: a slot's heads must be contiguous and of q's size, and the caches hold every sequence")
    return shape, stride


def _vector(t, n: int, name: str) -> None:
    """An int32 vector on the device with an entry for each of n."""
    if t.dtype is not torch.int32:
        _need(t, torch.int32, name)
    if t.dim() != 1 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous vector of at least {n} entries")


def _workspace(side, workspace, need: int, device):
    """Scratch for a call that was given none, or none that it can use."""
    if workspace is not None:
        raise ValueError("workspace: expected a contiguous tensor")
    return _scratch(side, torch.empty, max(need, 16), dtype=torch.uint8, device=device)


def _attn_decode_window(q, k_cache, v_cache, kv_len, out, workspace, split_len, window, sinks, scale, stream):
    _rows_of(q, out, "attn_decode")
    bsz, hq, d = q.shape
    shape, stride = _window_caches(k_cache, v_cache, bsz, d, "attn_decode")
    _vector(kv_len, bsz, "kv_len")
    _window_ints(window, sinks)
    _here(("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("kv_len", kv_len), ("out", out), ("workspace", workspace))
    lmax = shape[1]
    side = None if stream is None else _side(stream)
    if out is None:
        out = _empty_like(side)(q)
    if workspace is None or not workspace.is_contiguous():
        workspace = _workspace(side, workspace, attn_decode_workspace(bsz, hq, d, lmax, split_len, window, sinks), q.device)
    if side is not None:
        _hold(side, q, k_cache, v_cache, kv_len, out, workspace)
    _check(lib().kinv_attn_decode_window(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), stride[0], stride[1],
                                         kv_len.data_ptr(), out.data_ptr(), bsz, hq, shape[2], d, lmax, split_len, window,
                                         sinks, scale, workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), _stream(stream)),
           "kinv_attn_decode_window")
    return out


def attn_decode(q, k_cache, v_cache, kv_len, out=None, workspace=None, split_len=SPLIT_LEN,
                scale: float = 0.0, stream=None, window: int = 0, sinks: int = 0):
    """q [B][Hq][D]; caches [B][Lmax][Hkv][D] (or any layout with the same
    last two dims and strides along B and L); kv_len int32 [B].  With a window a
    row sees its last ``window`` keys and the first ``sinks`` of its sequence."""
    if window or sinks < 0:
        return _attn_decode_window(q, k_cache, v_cache, kv_len, out, workspace, split_len, window, sinks, scale,
                                   stream)
    _need(q, torch.bfloat16, "q")
    _need(kv_len, torch.int32, "kv_len")
    bsz, hq, d = q.shape
    lmax, hkv = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = _empty_like(_side(stream))(q)
    need = attn_decode_workspace(bsz, hq, d, lmax, split_len)
    if workspace is None:
        workspace = _scratch(_side(stream), torch.empty, max(need, 16), dtype=torch.uint8, device=q.device)
    _check(lib().kinv_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.stride(0),
                                  k_cache.stride(1), _ptr(kv_len), _ptr(out), bsz, hq, hkv, d, lmax,
                                  split_len, float(scale), _ptr(workspace), workspace.numel(),
                                  _stream(stream)), "kinv_attn_decode")
    return out


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def attn_decode_noalloc(q, k_cache, v_cache, kv_len, out, split_len=SPLIT_LEN, scale: float = 0.0,
                        stream=None):
    """Decode attention for callers that cannot allocate device memory: the
    library's own scratch array holds the partials (up to
    NOALLOC_SCRATCH_BYTES; calls sharing a device must not overlap on the GPU).
    ``out`` must be given, since this path allocates nothing."""
    _need(q, torch.bfloat16, "q")
    _need(k_cache, torch.bfloat16, "k_cache")
    _need(v_cache, torch.bfloat16, "v_cache")
    _need(kv_len, torch.int32, "kv_len")
    _need(out, torch.bfloat16, "out")
    if tuple(out.shape) != tuple(q.shape) or not out.is_contiguous() or not q.is_contiguous():
        raise ValueError("attn_decode_noalloc: q and out must be contiguous [B][Hq][D] of one shape")
    if tuple(v_cache.shape) != tuple(k_cache.shape) or v_cache.stride() != k_cache.stride():
        raise ValueError("attn_decode_noalloc: the caches must share shape and strides")
    bsz, hq, d = q.shape
    lmax, hkv = k_cache.shape[1], k_cache.shape[2]
    _check(lib().kinv_attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.stride(0),
                                          k_cache.stride(1), _ptr(kv_len), _ptr(out), bsz, hq, hkv,
                                          d, lmax, split_len, float(scale), _stream(stream)),
           "kinv_attn_decode_noalloc")
    return out


def attn_prefill_workspace(total_rows: int, n_q: int, head_dim: int, max_kv: int,
                           split_len: int = SPLIT_LEN) -> int:
    return int(lib().kinv_attn_prefill_workspace(total_rows, n_q, head_dim, max_kv, split_len))


def attn_prefill_window_workspace(batch: int, max_q_len: int, n_q: int, n_kv: int, head_dim: int, max_kv: int,
                                  window: int = 0, sinks: int = 0, split_len: int = SPLIT_LEN) -> int:
    """Bytes with which attn_prefill with a window spreads short chunks over the whole
    GPU (the bits are the same without); 0 where it would not help."""
    return int(lib().kinv_attn_prefill_window_workspace(batch, max_q_len, n_q, n_kv, head_dim, max_kv, split_len, window,
                                                        sinks))


def _attn_prefill_window(q, k_cache, v_cache, q_start, q_len, q_offset, max_q_len, max_kv, out, workspace,
                         split_len, window, sinks, scale, stream):
    _rows_of(q, out, "attn_prefill")
    rows, hq, d = q.shape
    bsz = q_start.shape[0]
    shape, stride = _window_caches(k_cache, v_cache, bsz, d, "attn_prefill")
    if max_kv > shape[1]:
        raise ValueError("attn_prefill: the caches are smaller than max_kv")
    _vector(q_start, bsz, "q_start")
    _vector(q_len, bsz, "q_len")
    _vector(q_offset, bsz, "q_offset")
    _window_ints(window, sinks)
    _here(("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("q_start", q_start), ("q_len", q_len),
          ("q_offset", q_offset), ("out", out), ("workspace", workspace))
    side = None if stream is None else _side(stream)
    if out is None:
        out = _empty_like(side)(q)
    if workspace is None or not workspace.is_contiguous():
        need = attn_prefill_window_workspace(bsz, max_q_len, hq, shape[2], d, max_kv, window, sinks, split_len)
        workspace = _workspace(side, workspace, need, q.device) if need or workspace is not None else None
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if side is not None:
        _hold(side, q, k_cache, v_cache, q_start, q_len, q_offset, out, workspace)
    _check(lib().kinv_attn_prefill_window(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), stride[0], stride[1],
                                          q_start.data_ptr(), q_len.data_ptr(), q_offset.data_ptr(), out.data_ptr(),
                                          bsz, rows, max_q_len, max_kv, hq, shape[2], d, split_len, window, sinks, scale,
                                          ws, ws_bytes, _stream(stream)), "kinv_attn_prefill_window")
    return out


def attn_prefill(q, k_cache, v_cache, q_start, q_len, q_offset, max_q_len: int, max_kv: int,
                 out=None, workspace=None, split_len=SPLIT_LEN, scale: float = 0.0, stream=None,
                 window: int = 0, sinks: int = 0):
    """q [rows][Hq][D]; per-sequence int32 q_start, q_len, q_offset [B].  With a
    window a row sees its last ``window`` keys and the first ``sinks`` of its
    sequence; rows of no sequence are not written."""
    if window or sinks < 0:
        return _attn_prefill_window(q, k_cache, v_cache, q_start, q_len, q_offset, max_q_len, max_kv, out, workspace,
                                    split_len, window, sinks, scale, stream)
    _need(q, torch.bfloat16, "q")
    rows, hq, d = q.shape
    hkv = k_cache.shape[2]
    bsz = q_start.shape[0]
    if out is None:
        out = _empty_like(_side(stream))(q)
    need = attn_prefill_workspace(rows, hq, d, max_kv, split_len)
    if workspace is None:
        workspace = _scratch(_side(stream), torch.empty, max(need, 16), dtype=torch.uint8, device=q.device)
    _check(lib().kinv_attn_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.stride(0),
                                   k_cache.stride(1), _ptr(q_start), _ptr(q_len), _ptr(q_offset),
                                   _ptr(out), bsz, rows, max_q_len, max_kv, hq, hkv, d, split_len,
                                   float(scale), _ptr(workspace), workspace.numel(),
                                   _stream(stream)), "kinv_attn_prefill")
    return out


# -------------------------------------------------------- 8-bit key/value cache
CACHE8_DTYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


class Cache8Struct(ctypes.Structure):
    """kinv_cache8: an 8-bit key/value cache."""
    _fields_ = [("k", _c_p), ("v", _c_p), ("k_exp", _c_p), ("v_exp", _c_p), ("seq_stride", _i64),
                ("tok_stride", _i64), ("exp_seq_stride", _i64), ("exp_head_stride", _i64), ("B", _i32),
                ("slots", _i32), ("dtype", _i32)]


class Cache8:
    """Keys and values as 8-bit codes with a power-of-two scale for every (token,
    kv head): codes k, v [B][slots][Hkv][D] (torch.float8_e4m3fn or torch.int8), and
    exponents k_exp, v_exp [B][Hkv][slots] (int8); a value is code * 2^exponent, an
    exponent of -128 marks a vector of NaN.  Holds its tensors."""

    def __init__(self, k, v, k_exp, v_exp):
        if k.dtype not in CACHE8_DTYPES.values():
            raise TypeError(f"k: expected torch.float8_e4m3fn or torch.int8, got {k.dtype}")
        for t, dt, name in ((k, k.dtype, "k"), (v, k.dtype, "v"), (k_exp, torch.int8, "k_exp"),
                            (v_exp, torch.int8, "v_exp")):
            _need(t, dt, name)
            if t.device != k.device:
                raise ValueError(f"Cache8: {name} is on {t.device}, k on {k.device}")
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride():
            raise ValueError("Cache8: the codes must be [B][slots][Hkv][D] and share shape and strides")
        bsz, slots, hkv, d = k.shape
        s0, s1, s2, s3 = k.stride()
        if s3 != 1 or (s2 != d and hkv > 1):
            raise ValueError("Cache8: a slot's heads must be contiguous")
        if tuple(k_exp.shape) != (bsz, hkv, slots) or v_exp.shape != k_exp.shape or v_exp.stride() != k_exp.stride() \
                or (k_exp.stride(2) != 1 and slots > 1):
            raise ValueError("Cache8: the exponents must be [B][Hkv][slots], a head's slots contiguous")
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.B, self.slots, self.n_kv, self.head_dim, self.device = bsz, slots, hkv, d, k.device
        self.struct = Cache8Struct(_ptr(k), _ptr(v), _ptr(k_exp), _ptr(v_exp), s0, s1, k_exp.stride(0),
                                   k_exp.stride(1), bsz, slots, I8 if k.dtype == torch.int8 else E4M3)
        self.ptr = ctypes.byref(self.struct)
        self.tensors = (k, v, k_exp, v_exp)

    @classmethod
    def empty(cls, batch: int, slots: int, n_kv: int, head_dim: int, dtype: str = "e4m3", device="cuda"):
        """A cache whose every value is 0; dtype "e4m3" or "int8"."""
        if dtype not in CACHE8_DTYPES:
            raise ValueError(f"dtype: expected one of {sorted(CACHE8_DTYPES)}, got {dtype!r}")
        k, v = (torch.zeros(batch, slots, n_kv, head_dim, dtype=torch.uint8, device=device).view(CACHE8_DTYPES[dtype])
                for _ in range(2))
        ke, ve = (torch.zeros(batch, n_kv, slots, dtype=torch.int8, device=device) for _ in range(2))
        return cls(k, v, ke, ve)

    def sequences(self, first: int, last: int) -> "Cache8":
        """Sequences first .. last - 1 of the same memory."""
        return Cache8(*(t[first:last] for t in self.tensors))


def rope_append8(qkv, q_out, cache: Cache8, seq, pos, n_q, n_kv, head_dim, rope_base, q_norm=None, k_norm=None,
                 eps=1e-6, stream=None):
    """rope_append with the keys and values of the rows quantised into ``cache`` at
    [seq][pos]; q_out [rows][Hq][D].  A row outside the cache is left out (its q_out
    too) and recorded in the device status; no two rows may name one place."""
    bf = torch.bfloat16
    if not qkv.dtype is q_out.dtype is bf:
        _need(qkv, bf, "qkv")
        _need(q_out, bf, "q_out")
    (rows, width), (ld, step) = qkv.shape, qkv.stride()
    if (step != 1 or width != (n_q + 2 * n_kv) * head_dim or not q_out.is_contiguous()
            or q_out.numel() < rows * n_q * head_dim or cache.n_kv != n_kv or cache.head_dim != head_dim):
        raise ValueError("rope_append8: shapes or layouts do not match")
    _vector(seq, rows, "seq")
    _vector(pos, rows, "pos")
    for t, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if t is not None and not (t.dtype is bf and t.is_contiguous() and t.numel() >= head_dim):
            _need(t, bf, name)
            raise ValueError(f"rope_append8: {name} must hold a contiguous gain for each of a head's values")
    _here(("qkv", qkv), ("q_out", q_out), ("cache", cache.k), ("seq", seq), ("pos", pos), ("q_norm", q_norm),
          ("k_norm", k_norm))
    if stream is not None and (side := _side(stream)) is not None:
        _hold(side, qkv, q_out, seq, pos, q_norm, k_norm, *cache.tensors)
    _check(lib().kinv_rope_append8(qkv.data_ptr(), ld if rows > 1 else max(ld, width), q_out.data_ptr(), cache.ptr,
                                   seq.data_ptr(), pos.data_ptr(), _ptr(q_norm), _ptr(k_norm), eps, rows, n_q, n_kv,
                                   head_dim, rope_base, _stream(stream)), "kinv_rope_append8")
    return q_out


def _tokens(k, v, cache: Cache8, what: str):
    """Shape and strides of bf16 k, v [B][n][Hkv][D] that go into or come out of ``cache``."""
    bf = torch.bfloat16
    if not k.dtype is v.dtype is bf:
        _need(k, bf, "k")
        _need(v, bf, "v")
    shape, stride = k.shape, k.stride()
    if len(shape) != 4 or v.shape != shape or v.stride() != stride:
        raise ValueError(f"{what}: k and v must be [B][n][Hkv][D] and share shape and strides")
    bsz, n, hkv, d = shape
    if hkv != cache.n_kv or d != cache.head_dim or bsz > cache.B or stride[3] != 1 or (stride[2] != d and hkv > 1):
        raise ValueError(f"{what}: k and v must match the cache's heads and sequences, a token's heads contiguous")
    return bsz, n, stride[0], stride[1] if n > 1 else hkv * d


def cache8_write(cache: Cache8, k, v, start, length, stream=None) -> None:
    """bf16 k, v [B][n][Hkv][D] into ``cache``: token i < length[b] of sequence b goes
    to slot start[b] + i (int32 [B], device).  A sequence that does not fit is left
    out and recorded in the device status."""
    bsz, n, s0, s1 = _tokens(k, v, cache, "cache8_write")
    _vector(start, bsz, "start")
    _vector(length, bsz, "length")
    _here(("k", k), ("v", v), ("cache", cache.k), ("start", start), ("length", length))
    if stream is not None and (side := _side(stream)) is not None:
        _hold(side, k, v, start, length, *cache.tensors)
    _check(lib().kinv_cache8_write(k.data_ptr(), v.data_ptr(), s0, s1, cache.ptr, start.data_ptr(), length.data_ptr(),
                                   bsz, n, cache.n_kv, cache.head_dim, _stream(stream)), "kinv_cache8_write")


def cache8_read(cache: Cache8, start, length, n: int = 0, k=None, v=None, stream=None):
    """The reverse: (k, v) bf16 [B][n][Hkv][D] whose token i < length[b] is slot
    start[b] + i (n bounds length).  Tokens from length[b] on, and those of a
    sequence left out, keep what the given k and v held; where they are allocated
    here they hold anything."""
    side = None if stream is None else _side(stream)
    if k is None and v is None:
        hkv, d = cache.n_kv, cache.head_dim
        bsz, s1 = start.shape[0], hkv * d
        s0 = n * s1
        if bsz > cache.B:
            raise ValueError("cache8_read: more sequences than the cache's")
        k = _empty(side)((bsz, n, hkv, d), dtype=torch.bfloat16, device=cache.device)
        v = _empty_like(side)(k)
    elif k is None or v is None:
        raise ValueError("cache8_read: k and v are given together")
    else:
        bsz, n, s0, s1 = _tokens(k, v, cache, "cache8_read")
    _vector(start, bsz, "start")
    _vector(length, bsz, "length")
    _here(("k", k), ("v", v), ("cache", cache.k), ("start", start), ("length", length))
    if side is not None:
        _hold(side, k, v, start, length, *cache.tensors)
    _check(lib().kinv_cache8_read(cache.ptr, start.data_ptr(), length.data_ptr(), k.data_ptr(), v.data_ptr(), s0, s1,
                                  bsz, n, cache.n_kv, cache.head_dim, _stream(stream)), "kinv_cache8_read")
    return k, v


def attn_decode8_workspace(batch: int, n_q: int, head_dim: int, slots: int, window: int = 0, sinks: int = 0,
                           split_len: int = SPLIT_LEN) -> int:
    return int(lib().kinv_attn_decode8_workspace(batch, n_q, head_dim, slots, window, sinks, split_len))


def attn_decode8(q, cache: Cache8, kv_len, out=None, workspace=None, window: int = 0, sinks: int = 0,
                 split_len=SPLIT_LEN, scale: float = 0.0, stream=None):
    """attn_decode over an 8-bit cache: q [B][Hq][D], kv_len int32 [B].  With a window
    a row sees its last ``window`` keys and the first ``sinks`` of its sequence.  A row
    has the bits of attn_decode on the cache read back."""
    _rows_of(q, out, "attn_decode8")
    bsz, hq, d = q.shape
    if d != cache.head_dim:
        raise ValueError("attn_decode8: q's heads are not of the cache's size")
    _vector(kv_len, bsz, "kv_len")
    _window_ints(window, sinks)
    _here(("q", q), ("cache", cache.k), ("kv_len", kv_len), ("out", out), ("workspace", workspace))
    side = None if stream is None else _side(stream)
    if out is None:
        out = _empty_like(side)(q)
    if workspace is None or not workspace.is_contiguous():
        workspace = _workspace(side, workspace, attn_decode8_workspace(bsz, hq, d, cache.slots, window, sinks, split_len),
                               q.device)
    if side is not None:
        _hold(side, q, out, kv_len, workspace, *cache.tensors)
    _check(lib().kinv_attn_decode8(q.data_ptr(), cache.ptr, kv_len.data_ptr(), out.data_ptr(), bsz, hq, cache.n_kv, d,
                                   split_len, window, sinks, scale, workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "kinv_attn_decode8")
    return out


def attn_prefill8_workspace(batch: int, total_rows: int, n_q: int, n_kv: int, head_dim: int, max_kv: int,
                            split_len: int = SPLIT_LEN, max_q_len=None, window: int = 0, sinks: int = 0) -> int:
    """Bytes for attn_prefill8: with max_q_len, for a call of that bound, window and
    sinks; without, enough for every window and every chunk of up to total_rows (1.6 GB
    behind 131,072 keys of 32/8 heads of 128, of which a 4,096-key window needs 0.6)."""
    most = int(lib().kinv_attn_prefill8_workspace(batch, total_rows, n_q, n_kv, head_dim, max_kv, split_len))
    if max_q_len is None or not most:
        return most
    rows = min(max_q_len, total_rows, max_kv)
    return batch * max_kv * n_kv * head_dim * 4 + attn_prefill_window_workspace(batch, rows, n_q, n_kv, head_dim, max_kv,
                                                                                window, sinks, split_len)


def attn_prefill8(q, cache: Cache8, q_start, q_len, q_offset, max_q_len: int, max_kv: int, out=None, workspace=None,
                  window: int = 0, sinks: int = 0, split_len=SPLIT_LEN, scale: float = 0.0, stream=None):
    """attn_prefill over an 8-bit cache, which already holds the rows' keys and
    values: q [rows][Hq][D]; per-sequence int32 q_start, q_len, q_offset [B].  Rows of
    no sequence are not written."""
    _rows_of(q, out, "attn_prefill8")
    rows, hq, d = q.shape
    bsz = q_start.shape[0]
    if d != cache.head_dim:
        raise ValueError("attn_prefill8: q's heads are not of the cache's size")
    _vector(q_start, bsz, "q_start")
    _vector(q_len, bsz, "q_len")
    _vector(q_offset, bsz, "q_offset")
    _window_ints(window, sinks)
    _here(("q", q), ("cache", cache.k), ("q_start", q_start), ("q_len", q_len), ("q_offset", q_offset), ("out", out),
          ("workspace", workspace))
    side = None if stream is None else _side(stream)
    if out is None:
        out = _empty_like(side)(q)
    if workspace is None or not workspace.is_contiguous():
        need = attn_prefill8_workspace(bsz, rows, hq, cache.n_kv, d, max_kv, split_len, max_q_len, window, sinks)
        workspace = _workspace(side, workspace, need, q.device)
    if side is not None:
        _hold(side, q, out, q_start, q_len, q_offset, workspace, *cache.tensors)
    _check(lib().kinv_attn_prefill8(q.data_ptr(), cache.ptr, q_start.data_ptr(), q_len.data_ptr(), q_offset.data_ptr(),
                                    out.data_ptr(), bsz, rows, max_q_len, max_kv, hq, cache.n_kv, d, split_len, window,
                                    sinks, scale, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "kinv_attn_prefill8")
    return out


# --------------------------------------------------- trees of drafted tokens
TREE_MAX_NODES = 64
MARK_COUNT, MARK_PATH, MARK_TOKENS = 1, 2, 4


class TreeStruct(ctypes.Structure):
    """kinv_tree: a batch of trees of drafted tokens."""
    _fields_ = [("ctx_len", _c_p), ("n_nodes", _c_p), ("row_offset", _c_p), ("parent", _c_p),
                ("B", _i32), ("total_rows", _i32), ("max_nodes", _i32), ("max_kv", _i32)]


class Tree:
    """A batch of trees of drafted tokens over device int32 tensors (kept while
    the tree is used): ctx_len, n_nodes, row_offset [B], parent [total_rows]
    (index of the parent within the sequence, or -1).  Node i of sequence b is
    row row_offset[b] + i, sits in cache slot ctx_len[b] + i and has position
    ctx_len[b] + its depth.  max_nodes bounds n_nodes, max_kv bounds ctx_len +
    n_nodes (the cache's slots).  The tensors may be refilled between calls."""

    def __init__(self, ctx_len, n_nodes, row_offset, parent, max_nodes: int, max_kv: int):
        for t, name in ((ctx_len, "ctx_len"), (n_nodes, "n_nodes"), (row_offset, "row_offset"),
                        (parent, "parent")):
            _need(t, torch.int32, name)
            if t.dim() != 1 or not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous vector")
        b = ctx_len.shape[0]
        if n_nodes.shape[0] != b or row_offset.shape[0] != b:
            raise ValueError("Tree: ctx_len, n_nodes and row_offset must have one entry per sequence")
        self.tensors = (ctx_len, n_nodes, row_offset, parent)
        self.B, self.total_rows, self.max_nodes, self.max_kv = b, parent.shape[0], int(max_nodes), int(max_kv)
        self.struct = TreeStruct(_ptr(ctx_len), _ptr(n_nodes), _ptr(row_offset), _ptr(parent), b,
                                 self.total_rows, self.max_nodes, self.max_kv)
        self.ptr = ctypes.byref(self.struct)


def _tree_cache(k_cache, v_cache, tree: Tree, what: str):
    """Shape and strides of the caches [B][slots][Hkv][D], which hold the
    tree's sequences and max_kv slots each."""
    shape, stride = k_cache.shape, k_cache.stride()
    if v_cache.shape != shape or v_cache.stride() != stride:
        raise ValueError(f"{what}: the caches must share shape and strides")
    bsz, slots, _, d = shape
    if stride[3] != 1 or stride[2] != d:
        raise ValueError(f"{what}: a slot's heads must be contiguous")
    if bsz < tree.B or slots < tree.max_kv:
        raise ValueError(f"{what}: the caches are smaller than the tree's sequences and max_kv")
    return shape, stride


def rope_append_tree(qkv, q_out, k_cache, v_cache, tree: Tree, n_q, n_kv, head_dim, rope_base,
                     q_norm=None, k_norm=None, eps=1e-6, stream=None):
    """kinv_rope_append for the rows of drafted trees: qkv [rows][(Hq + 2 Hkv) D]
    rotated by each node's position -> q_out [rows][Hq][D], keys and values into
    the caches [B][slots][Hkv][D] at the node's slot."""
    bf = torch.bfloat16
    if not (qkv.dtype is q_out.dtype is k_cache.dtype is v_cache.dtype is bf and qkv.is_cuda and q_out.is_cuda
            and k_cache.is_cuda and v_cache.is_cuda):
        for t, name in ((qkv, "qkv"), (q_out, "q_out"), (k_cache, "k_cache"), (v_cache, "v_cache")):
            _need(t, bf, name)
    shape, stride = _tree_cache(k_cache, v_cache, tree, "rope_append_tree")
    (rows, width), (ld, step) = qkv.shape, qkv.stride()
    if (rows < tree.total_rows or step != 1 or not q_out.is_contiguous() or width != (n_q + 2 * n_kv) * head_dim
            or q_out.numel() < tree.total_rows * n_q * head_dim or shape[2] != n_kv or shape[3] != head_dim):
        raise ValueError("rope_append_tree: shapes or layouts do not match")
    for t, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if t is not None and not (t.dtype is bf and t.is_cuda and t.is_contiguous() and t.numel() >= head_dim):
            _need(t, bf, name)
            raise ValueError(f"rope_append_tree: {name} must hold a contiguous gain for each of a head's values")
    side = _side(stream)
    if side is not None:
        _hold(side, qkv, q_out, k_cache, v_cache, q_norm, k_norm, *tree.tensors)
    _check(lib().kinv_rope_append_tree(qkv.data_ptr(), ld, q_out.data_ptr(), k_cache.data_ptr(),
                                       v_cache.data_ptr(), stride[0], stride[1], tree.ptr, _ptr(q_norm),
                                       _ptr(k_norm), eps, n_q, n_kv, head_dim, rope_base, _stream(stream)),
           "kinv_rope_append_tree")
    return q_out


def attn_tree_workspace(tree: Tree, n_q: int, n_kv: int, head_dim: int, split_len: int = SPLIT_LEN) -> int:
    return int(lib().kinv_attn_tree_workspace(tree.B, tree.total_rows, tree.max_nodes, n_q, n_kv, head_dim,
                                              tree.max_kv, split_len))


def attn_tree(q, k_cache, v_cache, tree: Tree, out=None, workspace=None, split_len=SPLIT_LEN,
              scale: float = 0.0, stream=None):
    """q [rows][Hq][D]; caches [B][slots][Hkv][D], which already hold the
    nodes' keys and values in their slots.  Each row has the bits of attn_decode
    behind the context and the node's path.  Rows of no sequence, and those of a
    sequence left out for its broken tree, are not written: they hold what ``out``
    held, anything where it is not given."""
    side = _side(stream)
    if out is None:
        out = _empty_like(side)(q)
    bf = torch.bfloat16
    if not (q.dtype is out.dtype is k_cache.dtype is v_cache.dtype is bf and q.is_cuda and out.is_cuda
            and k_cache.is_cuda and v_cache.is_cuda):
        for t, name in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (out, "out")):
            _need(t, bf, name)
    shape, stride = _tree_cache(k_cache, v_cache, tree, "attn_tree")
    rows, hq, d = q.shape
    hkv = shape[2]
    if (not q.is_contiguous() or not out.is_contiguous() or rows < tree.total_rows
            or out.shape != q.shape or shape[3] != d):
        raise ValueError("attn_tree: shapes or layouts do not match")
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace: expected a CUDA tensor")
    if workspace is None:
        workspace = _scratch(side, torch.empty, max(attn_tree_workspace(tree, hq, hkv, d, split_len), 16),
                             dtype=torch.uint8, device=q.device)
    if side is not None:
        _hold(side, q, k_cache, v_cache, out, workspace, *tree.tensors)
    _check(lib().kinv_attn_tree(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), stride[0], stride[1],
                                tree.ptr, out.data_ptr(), hq, hkv, d, split_len, scale, workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream(stream)),
           "kinv_attn_tree")
    return out


def tree_accept(tree: Tree, tokens, next_tokens, kv=None, n_accepted=None, path=None, out_tokens=None,
                stream=None):
    """The path of drafted nodes that the model's own tokens agree with, moved
    to its place in the cache.  tokens, next_tokens: int32 [rows] (a node's
    token, the model's token after it); kv: [layers][2][B][slots][Hkv][D] bf16,
    changed in place (None: only the path is found).  Returns (n_accepted [B],
    path [B][max_nodes], out_tokens [B][max_nodes]) int32.  For a sequence left out
    for its broken tree those that are allocated here say 0 nodes and -1; those
    that are given keep what they held."""
    b, n, i32 = tree.B, tree.max_nodes, torch.int32
    side = _side(stream)
    empty = _empty(side)
    mark = 0    # results that are allocated here are defined for a sequence left out, too
    given = [(tokens, "tokens", tree.total_rows), (next_tokens, "next_tokens", tree.total_rows)]
    if n_accepted is None:
        mark |= MARK_COUNT
        n_accepted = empty(b, dtype=i32, device=tokens.device)
    else:
        given.append((n_accepted, "n_accepted", b))
    if path is None:
        mark |= MARK_PATH
        path = empty(b, n, dtype=i32, device=tokens.device)
    else:
        given.append((path, "path", b * n))
    if out_tokens is None:
        mark |= MARK_TOKENS
        out_tokens = empty(b, n, dtype=i32, device=tokens.device)
    else:
        given.append((out_tokens, "out_tokens", b * n))
    for t, name, least in given:
        if t.dtype is not i32 or not t.is_cuda:
            _need(t, i32, name)
        if t.numel() < least or not t.is_contiguous():
            raise ValueError(f"tree_accept: {name} must be contiguous with at least {least} entries")
    if kv is None:
        kp = vp = None
        layers = ls = ss = ts = hkv = d = 0
    else:
        _need(kv, torch.bfloat16, "kv")
        layers, two, bsz, slots, hkv, d = kv.shape
        ls, cs, ss, ts, hs, es = kv.stride()
        if two != 2 or bsz < b or slots < tree.max_kv or es != 1 or hs != d:
            raise ValueError("tree_accept: kv must be [layers][2][B][slots][Hkv][D] with room for the tree")
        kp = kv.data_ptr()
        vp = kp + 2 * cs
    if side is not None:
        _hold(side, tokens, next_tokens, kv, n_accepted, path, out_tokens, *tree.tensors)
    _check(lib().kinv_tree_accept_marked(tree.ptr, tokens.data_ptr(), next_tokens.data_ptr(), kp, vp, layers, ls, ss,
                                         ts, hkv, d, n_accepted.data_ptr(), path.data_ptr(), out_tokens.data_ptr(),
                                         mark, _stream(stream)), "kinv_tree_accept")
    return n_accepted, path, out_tokens


# --------------------------------------------------------- log probabilities
def logprobs(logits, ids=None, top_k: int = 0, stream=None):
    """logits fp32 or bf16 [rows][V]; ids int32 [rows][n] (negative: padding).
    Returns (logprobs fp32 [rows][n] or None, entropy fp32 [rows], top_ids int32
    [rows][top_k] or None, top_logprobs fp32 [rows][top_k] or None)."""
    dt = logits.dtype
    if dt is not torch.float32 and dt is not torch.bfloat16:
        raise TypeError(f"logits: expected torch.float32 or torch.bfloat16, got {dt}")
    _need(logits, dt, "logits")
    (rows, v), (ld, step) = logits.shape, logits.stride()
    if step != 1 and v > 1:
        raise ValueError("logprobs: the ids of a row must be contiguous")
    dev, side = logits.device, _side(stream)
    empty = _empty(side)
    n_ids, lp, lp_ptr, ids_ptr = 0, None, None, None
    if ids is not None:
        _need(ids, torch.int32, "ids")
        if ids.dim() != 2 or ids.shape[0] != rows or not ids.is_contiguous():
            raise ValueError("logprobs: ids must be a contiguous [rows][n]")
        n_ids = ids.shape[1]
        lp = empty(rows, n_ids, dtype=torch.float32, device=dev)
        lp_ptr, ids_ptr = lp.data_ptr(), ids.data_ptr()
    entropy = empty(rows, dtype=torch.float32, device=dev)
    top_ids = top_lp = top_ptr = top_lp_ptr = None
    if top_k:
        top_ids = empty(rows, top_k, dtype=torch.int32, device=dev)
        top_lp = empty(rows, top_k, dtype=torch.float32, device=dev)
        top_ptr, top_lp_ptr = top_ids.data_ptr(), top_lp.data_ptr()
    if side is not None:
        _hold(side, logits, ids)
    _check(lib().kinv_logprobs(logits.data_ptr(), F32 if dt is torch.float32 else BF16,
                               ld if rows > 1 else max(ld, v), rows, v, ids_ptr, n_ids, lp_ptr,
                               entropy.data_ptr(), top_k, top_ptr, top_lp_ptr, _stream(stream)), "kinv_logprobs")
    return lp, entropy, top_ids, top_lp


# ------------------------------------------------------------------ sampler
@dataclass
class SamplingParams:
    """Per-request sampler settings (the fields a Kinetic receipt records)."""
    temperature: float = 0.8
    top_k: int = 50
    top_p: float = 0.95
    min_p: float = 0.05
    repeat_penalty: float = 1.1
    repeat_last_n: int = 64
    seed: int = 42
    presence_penalty: float = 0.0
    frequency_penalty: float = 0.0
    logit_bias: dict = None   # {id: bias}, applied in insertion order
    typical_p: float = 1.0    # on when 0 < typical_p < 1


def sampling_params_device(params_list, device="cuda"):
    """kinv_sampling_params [B] packed on the device, and the device buffer
    of logit-bias entries they point to (None without any); keep both alive
    while sampling with them."""
    from . import synth
    entries, _ = synth.bias_entries(params_list)
    bias = torch.from_numpy(entries.view(np.uint8).copy()).to(device) if len(entries) else None
    packed = synth.sampling_struct(params_list, bias.data_ptr() if bias is not None else 0)
    return torch.from_numpy(packed.view(np.uint8).copy()).to(device), bias


def sample(logits, params_dev, history, hist_len, step, out=None, stream=None):
    """logits fp32 [B][V]; params_dev uint8 tensor holding B packed
    kinv_sampling_params; history int32 [B][H]; hist_len int32 [B];
    step int64 [B] -> int32 [B]."""
    _need(logits, torch.float32, "logits")
    bsz, v = logits.shape
    if out is None:
        out = _empty(_side(stream))(bsz, dtype=torch.int32, device=logits.device)
    _check(lib().kinv_sample(_ptr(logits), logits.stride(0), bsz, v, _ptr(params_dev),
                             _ptr(history), history.shape[1] if history is not None else 0,
                             _ptr(hist_len), _ptr(step), _ptr(out), None, 0, _stream(stream)),
           "kinv_sample")
    return out


# --------------------------------------------------------------------- glue
def embed(table, ids, out=None, stream=None):
    vocab, dim = table.shape
    rows = ids.shape[0]
    if out is None:
        out = _empty(_side(stream))(rows, dim, dtype=table.dtype, device=table.device)
    _check(lib().kinv_embed(_ptr(table), vocab, dim, _ptr(ids), _ptr(out), rows, _stream(stream)),
           "kinv_embed")
    return out


def add(x, y, out=None, stream=None):
    if out is None:
        out = _empty_like(_side(stream))(x)
    _check(lib().kinv_add(_ptr(x), _ptr(y), _ptr(out), x.numel(), _stream(stream)), "kinv_add")
    return out


def scale_columns(w, g, out=None, stream=None):
    """out[n][k] = bf16(w[n][k] * g[k]): a norm gain folded into a weight."""
    _need(w, torch.bfloat16, "w")
    _need(g, torch.bfloat16, "g")
    n, k = w.shape
    if out is None:
        out = _empty_like(_side(stream))(w)
    _check(lib().kinv_scale_columns(_ptr(w), w.stride(0), _ptr(g), _ptr(out), out.stride(0), n, k,
                                    _stream(stream)), "kinv_scale_columns")
    return out


def swiglu(gu, out=None, stream=None):
    rows, two_f = gu.shape
    f = two_f // 2
    if out is None:
        out = _empty(_side(stream))(rows, f, dtype=gu.dtype, device=gu.device)
    _check(lib().kinv_swiglu(_ptr(gu), gu.stride(0), _ptr(out), out.stride(0), rows, f,
                             _stream(stream)), "kinv_swiglu")
    return out


def rope_append(qkv, q_out, k_cache, v_cache, seq, pos, n_q, n_kv, head_dim, rope_base,
                q_norm=None, k_norm=None, eps=1e-6, stream=None):
    rows = qkv.shape[0]
    _check(lib().kinv_rope_append(_ptr(qkv), qkv.stride(0), _ptr(q_out), _ptr(k_cache),
                                  _ptr(v_cache), k_cache.stride(0), k_cache.stride(1), _ptr(seq),
                                  _ptr(pos), _ptr(q_norm), _ptr(k_norm), float(eps), rows, n_q,
                                  n_kv, head_dim, float(rope_base), _stream(stream)),
           "kinv_rope_append")
    return q_out


def decode_advance(tokens, history, hist_len, step, pos=None, kv_len=None, stream=None):
    bsz = tokens.shape[0]
    _check(lib().kinv_decode_advance(_ptr(tokens), _ptr(history), history.shape[1],
                                     _ptr(hist_len), _ptr(step), _ptr(pos), _ptr(kv_len), bsz,
                                     _stream(stream)), "kinv_decode_advance")


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
