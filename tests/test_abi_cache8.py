"""Host-side refusals of the 8-bit cache and windowed attention (no call here
reaches a device), the layout of kinv_cache8, and the workspace sizes."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from invariant_deterministic_gb300 import build, kinv
    build.build()
    return kinv


def _cache(lib, **kw):
    f = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, seq_stride=64 * 512, tok_stride=64, exp_seq_stride=512,
             exp_head_stride=512, B=2, slots=512, dtype=lib.I8)
    f.update(kw)
    return ctypes.byref(lib.Cache8Struct(**f))


def test_cache8_struct_layout(lib, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in lib.Cache8Struct._fields_]
    body = "".join(f'printf("%zu\\n", offsetof(kinv_cache8, {f}));' for f in names)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kinv.h"\nint main(void) {'
                   f'printf("%zu\\n%d\\n%d\\n", sizeof(kinv_cache8), KINV_E4M3, KINV_I8);{body}return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert out[:3] == [ctypes.sizeof(lib.Cache8Struct), lib.E4M3, lib.I8]
    assert out[3:] == [getattr(lib.Cache8Struct, f).offset for f in names]


def _append(lib, c, qkv=FAKE, ld=4 * 64, q=FAKE, seq=FAKE, pos=FAKE, eps=1e-6, rows=3, hq=2, hkv=1, d=64, base=1e4):
    return lib.lib().kinv_rope_append8(qkv, ld, q, c, seq, pos, None, None, eps, rows, hq, hkv, d, base, None)


def _write(lib, c, k=FAKE, v=FAKE, ss=64 * 10, ts=64, start=FAKE, length=FAKE, b=2, n=10, hkv=1, d=64):
    return lib.lib().kinv_cache8_write(k, v, ss, ts, c, start, length, b, n, hkv, d, None)


def _read(lib, c, k=FAKE, v=FAKE, ss=64 * 10, ts=64, start=FAKE, length=FAKE, b=2, n=10, hkv=1, d=64):
    return lib.lib().kinv_cache8_read(c, start, length, k, v, ss, ts, b, n, hkv, d, None)


def _decode8(lib, c, q=FAKE, n=FAKE, out=FAKE, b=2, hq=2, hkv=1, d=64, split=256, window=0, sinks=0, scale=0.0, ws=FAKE, wsb=1 << 30):
    return lib.lib().kinv_attn_decode8(q, c, n, out, b, hq, hkv, d, split, window, sinks, scale, ws, wsb, None)


def _prefill8(lib, c, q=FAKE, s=FAKE, n=FAKE, o=FAKE, out=FAKE, b=2, rows=20, most=10, kv=512, hq=2, hkv=1, d=64, split=256, window=0,
              sinks=0, ws=FAKE, wsb=1 << 30):
    return lib.lib().kinv_attn_prefill8(q, c, s, n, o, out, b, rows, most, kv, hq, hkv, d, split, window, sinks, 0.0, ws, wsb, None)


CALLS = [_append, _write, _read, _decode8, _prefill8]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("change,status", [
    (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(k_exp=None), "INVALID_ARG"), (dict(v_exp=None), "INVALID_ARG"),
    (dict(B=-1), "INVALID_ARG"), (dict(slots=-1), "INVALID_ARG"), (dict(dtype=0), "INVALID_ARG"), (dict(dtype=7), "INVALID_ARG"),
    (dict(tok_stride=32), "INVALID_ARG"), (dict(seq_stride=-16), "INVALID_ARG"), (dict(exp_seq_stride=-1), "INVALID_ARG"),
    (dict(k=FAKE + 8), "ALIGNMENT"), (dict(v=FAKE + 1), "ALIGNMENT"), (dict(tok_stride=72), "ALIGNMENT"), (dict(seq_stride=64 * 512 + 8), "ALIGNMENT")])
def test_bad_caches_are_refused_by_every_call(lib, call, change, status):
    assert call(lib, _cache(lib, **change)) == getattr(lib, "ERR_" + status)
    assert call(lib, None) == lib.ERR_INVALID_ARG


@pytest.mark.parametrize("call", CALLS)
def test_heads_are_refused_by_every_call(lib, call):
    assert call(lib, _cache(lib, tok_stride=96), d=96, **({"ld": 400} if call is _append else {})) == lib.ERR_UNSUPPORTED
    assert call(lib, _cache(lib, tok_stride=128, exp_head_stride=500), hkv=2) == lib.ERR_INVALID_ARG   # heads' exponents overlap
    assert call(lib, _cache(lib), hkv=0) == lib.ERR_INVALID_ARG
    if call in (_decode8, _prefill8):
        assert call(lib, _cache(lib), hq=3, hkv=1) == lib.ERR_UNSUPPORTED
        assert call(lib, _cache(lib, tok_stride=128), hq=3, hkv=2) == lib.ERR_INVALID_ARG
        assert call(lib, _cache(lib), split=128) == lib.ERR_UNSUPPORTED
        assert call(lib, _cache(lib), window=-1) == lib.ERR_INVALID_ARG
        assert call(lib, _cache(lib), sinks=-1) == lib.ERR_INVALID_ARG
        assert call(lib, _cache(lib), b=3) == lib.ERR_INVALID_ARG      # more than the cache's
        assert call(lib, _cache(lib), ws=None) == lib.ERR_INVALID_ARG
        assert call(lib, _cache(lib), ws=FAKE + 4) == lib.ERR_ALIGNMENT
        assert call(lib, _cache(lib), wsb=100) == lib.ERR_WORKSPACE
        assert call(lib, _cache(lib), q=FAKE + 2) == lib.ERR_ALIGNMENT
        assert call(lib, _cache(lib), out=None) == lib.ERR_INVALID_ARG


@pytest.mark.parametrize("change,status", [
    (dict(qkv=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(seq=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"),
    (dict(rows=-1), "INVALID_ARG"), (dict(hq=0), "INVALID_ARG"), (dict(base=0.0), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(ld=64), "INVALID_ARG"), (dict(ld=260), "ALIGNMENT"), (dict(qkv=FAKE + 2), "ALIGNMENT")])
def test_append_refusals(lib, change, status):
    assert _append(lib, _cache(lib), **change) == getattr(lib, "ERR_" + status)
    assert _append(lib, _cache(lib), rows=0) == lib.OK


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("change,status", [
    (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(start=None), "INVALID_ARG"), (dict(length=None), "INVALID_ARG"),
    (dict(b=-1), "INVALID_ARG"), (dict(b=3), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"), (dict(ts=32), "INVALID_ARG"), (dict(ss=-8), "INVALID_ARG"),
    (dict(ss=644), "ALIGNMENT"), (dict(ts=68), "ALIGNMENT"), (dict(k=FAKE + 2), "ALIGNMENT")])
def test_write_and_read_refusals(lib, call, change, status):
    assert call(lib, _cache(lib), **change) == getattr(lib, "ERR_" + status)
    assert call(lib, _cache(lib), b=0) == lib.OK and call(lib, _cache(lib), n=0) == lib.OK
    many = _cache(lib, tok_stride=64 * 2000, seq_stride=64 * 2000 * 512, exp_head_stride=512)
    assert call(lib, many, hkv=2000, ts=64 * 2000, ss=64 * 20000) == lib.ERR_UNSUPPORTED


def test_sequences_written_over_each_other_are_refused(lib):
    for change in (dict(seq_stride=0), dict(exp_seq_stride=0)):
        assert _append(lib, _cache(lib, **change)) == lib.ERR_INVALID_ARG
        assert _write(lib, _cache(lib, **change)) == lib.ERR_INVALID_ARG
    assert _read(lib, _cache(lib), ss=0) == lib.ERR_INVALID_ARG


def test_attention_refusals(lib):
    c = _cache(lib)
    assert _decode8(lib, c, n=None) == lib.ERR_INVALID_ARG and _decode8(lib, c, b=-1) == lib.ERR_INVALID_ARG
    assert _decode8(lib, c, b=0) == lib.OK
    assert _decode8(lib, _cache(lib, seq_stride=0)) == lib.ERR_INVALID_ARG
    for name in ("s", "n", "o"):
        assert _prefill8(lib, c, **{name: None}) == lib.ERR_INVALID_ARG
    assert _prefill8(lib, c, kv=513) == lib.ERR_INVALID_ARG          # more than the cache's slots
    assert _prefill8(lib, c, rows=0) == lib.OK and _prefill8(lib, c, most=0) == lib.OK and _prefill8(lib, c, b=0) == lib.OK
    assert _prefill8(lib, c, rows=-1) == lib.ERR_INVALID_ARG and _prefill8(lib, c, most=-1) == lib.ERR_INVALID_ARG
    wide = _cache(lib, tok_stride=512, seq_stride=512 * 512)
    assert _prefill8(lib, wide, most=2**31 - 1, rows=2**31 - 1, hq=64, hkv=8, wsb=2**40) == lib.ERR_UNSUPPORTED  # the number of tiles


def test_window_refusals(lib):
    L = lib.lib()

    def decode(window=5, sinks=1, d=64, hq=2, split=256, ws=FAKE, wsb=1 << 30, q=FAKE, n=FAKE):
        return L.kinv_attn_decode_window(q, FAKE, FAKE, 64 * 512, 64, n, FAKE, 2, hq, 1, d, 512, split, window, sinks, 0.0, ws, wsb, None)

    def prefill(window=5, sinks=1, d=64, hq=2, split=256, q=FAKE, rows=20, ws=None):
        return L.kinv_attn_prefill_window(q, FAKE, FAKE, 64 * 512, 64, FAKE, FAKE, FAKE, FAKE, 2, rows, 10, 512, hq, 1, d, split, window, sinks, 0.0,
                                          ws, 0, None)
    for call in (decode, prefill):
        assert call(window=-1) == lib.ERR_INVALID_ARG and call(sinks=-1) == lib.ERR_INVALID_ARG
        assert call(d=96) == lib.ERR_UNSUPPORTED and call(hq=3) == lib.ERR_UNSUPPORTED and call(split=128) == lib.ERR_UNSUPPORTED
        assert call(q=None) == lib.ERR_INVALID_ARG and call(q=FAKE + 2) == lib.ERR_ALIGNMENT
    assert decode(n=None) == lib.ERR_INVALID_ARG and decode(ws=None) == lib.ERR_INVALID_ARG and decode(wsb=100) == lib.ERR_WORKSPACE
    assert prefill(rows=0) == lib.OK and prefill(rows=-1) == lib.ERR_INVALID_ARG and prefill(ws=FAKE + 8) == lib.ERR_ALIGNMENT


def test_workspaces_grow_with_the_window(lib):
    full = lib.attn_decode_workspace(4, 32, 128, 32768)
    assert lib.attn_decode_workspace(4, 32, 128, 32768, window=10**6) == full
    assert lib.attn_decode8_workspace(4, 32, 128, 32768) == full
    one = lib.attn_decode_workspace(4, 32, 128, 256)
    for window, sinks, splits in ((1, 0, 1), (2, 0, 2), (257, 0, 2), (258, 0, 3), (1, 1, 2), (1, 257, 3), (4096, 4, 18)):
        # a window of W keys lies in at most (W + 254) / 256 + 1 splits
        want = lib.attn_decode_workspace(4, 32, 128, 256 * splits)
        assert lib.attn_decode_workspace(4, 32, 128, 32768, window=window, sinks=sinks) == want
        assert lib.attn_decode8_workspace(4, 32, 128, 32768, window, sinks) == want
    assert lib.attn_decode8_workspace(4, 32, 128, 100, 4096, 4) == one
    assert lib.attn_decode8_workspace(0, 32, 128, 100) == 0 and lib.attn_decode8_workspace(4, 32, 128, 100, -1) == 0
    # the keys and values read back, and the partials of 24 tiles over four splits
    assert lib.attn_prefill8_workspace(3, 10, 32, 8, 128, 1000) == 3 * 1000 * 8 * 128 * 4 + 24 * 4 * 128 * (128 + 2) * 4
    assert lib.attn_prefill8_workspace(3, 10, 32, 8, 128, 500) == 3 * 500 * 8 * 128 * 4
    for rows in (1, 32, 33, 128, 129, 4096):   # at most 38 tiles are spread
        bytes_of = lambda r: (r + 31) // 32 * 8 * 128 * 128 * (128 + 2) * 4
        assert lib.attn_prefill_window_workspace(1, rows, 32, 8, 128, 32768) == (bytes_of(rows) if rows <= 128 else 0)
        # over an 8-bit cache as much as any chunk of up to so many rows can use
        assert lib.attn_prefill8_workspace(1, rows, 32, 8, 128, 32768) == 32768 * 8 * 128 * 4 + bytes_of(min(rows, 128))
    # rows of a tile see 4,096 + 31 keys: 18 splits, and one of sinks
    assert lib.attn_prefill_window_workspace(1, 32, 32, 8, 128, 32768, 4096, 4) == 8 * 19 * 128 * (128 + 2) * 4
    assert lib.attn_prefill_window_workspace(5, 32, 32, 8, 128, 32768) == 0 and lib.attn_prefill_window_workspace(1, 32, 32, 8, 128, 512) == 0
    assert lib.attn_prefill8_workspace(3, 0, 32, 8, 128, 1000) == 0


def test_cache8_arguments(lib, monkeypatch):
    """The handle's own checks (the tensors' device check aside)."""
    monkeypatch.setattr(lib, "_need", lambda t, dt, name: None if t.dtype == dt else (_ for _ in ()).throw(TypeError(name)))
    k = torch.zeros(2, 10, 3, 64, dtype=torch.int8)
    e = torch.zeros(2, 3, 10, dtype=torch.int8)
    c = lib.Cache8(k, k.clone(), e, e.clone())
    assert (c.B, c.slots, c.n_kv, c.head_dim, c.struct.dtype) == (2, 10, 3, 64, lib.I8)
    assert c.sequences(1, 2).struct.k == k[1:].data_ptr() and c.sequences(1, 2).struct.B == 1
    with pytest.raises(TypeError):
        lib.Cache8(k.to(torch.uint8), k, e, e)
    with pytest.raises(TypeError):
        lib.Cache8(k, k.float(), e, e)
    for bad in ((k, k[:, :9], e, e), (k.transpose(2, 3), k.transpose(2, 3), e, e), (k, k, e[:, :2], e[:, :2]), (k, k, e[:, :, ::2], e[:, :, ::2]),
                (k[:, :, ::2], k[:, :, ::2], e[:, ::2], e[:, ::2])):
        with pytest.raises(ValueError):
            lib.Cache8(*bad)
    with pytest.raises(ValueError):
        lib.Cache8.empty(1, 10, 2, 64, "e5m2", device="cpu")
