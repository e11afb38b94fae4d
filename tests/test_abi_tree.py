"""Host-side refusals of the drafted-tree and log-probability calls (no call
here reaches a device), and the layout of kinv_tree."""
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


def _tree(lib, **kw):
    f = dict(ctx_len=FAKE, n_nodes=FAKE, row_offset=FAKE, parent=FAKE, B=2, total_rows=10, max_nodes=8, max_kv=512)
    f.update(kw)
    return ctypes.byref(lib.TreeStruct(**f))


def test_tree_struct_layout(lib, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in lib.TreeStruct._fields_]
    body = "".join(f'printf("%zu\\n", offsetof(kinv_tree, {f}));' for f in names)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kinv.h"\nint main(void) {'
                   f'printf("%zu\\n%d\\n", sizeof(kinv_tree), KINV_TREE_MAX_NODES);{body}return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert out[0] == ctypes.sizeof(lib.TreeStruct) and out[1] == lib.TREE_MAX_NODES
    assert out[2:] == [getattr(lib.TreeStruct, f).offset for f in names]


BAD_TREES = [
    (dict(B=-1), "INVALID_ARG"), (dict(total_rows=-1), "INVALID_ARG"), (dict(max_nodes=-1), "INVALID_ARG"),
    (dict(max_kv=-1), "INVALID_ARG"), (dict(max_nodes=65), "UNSUPPORTED"), (dict(B=65536), "UNSUPPORTED"),
    (dict(ctx_len=None), "INVALID_ARG"), (dict(n_nodes=None), "INVALID_ARG"),
    (dict(row_offset=None), "INVALID_ARG"), (dict(parent=None), "INVALID_ARG"),
]


def _rope(lib, t, qkv=FAKE, ld=4 * 64, q=FAKE, k=FAKE, v=FAKE, ss=64 * 512, ts=64, eps=1e-6, hq=2, hkv=1, d=64, base=1e4):
    return lib.lib().kinv_rope_append_tree(qkv, ld, q, k, v, ss, ts, t, None, None, eps, hq, hkv, d, base, None)


def _attn(lib, t, q=FAKE, k=FAKE, v=FAKE, ss=64 * 512, ts=64, out=FAKE, hq=2, hkv=1, d=64, split=256, ws=FAKE, wsb=1 << 30):
    return lib.lib().kinv_attn_tree(q, k, v, ss, ts, t, out, hq, hkv, d, split, 0.0, ws, wsb, None)


def _accept(lib, t, tok=FAKE, nxt=FAKE, k=FAKE, v=FAKE, layers=1, ls=64 * 1024, ss=64 * 512, ts=64, hkv=1, d=64, n=FAKE,
            path=FAKE, out=FAKE):
    return lib.lib().kinv_tree_accept(t, tok, nxt, k, v, layers, ls, ss, ts, hkv, d, n, path, out, None)


@pytest.mark.parametrize("change,status", BAD_TREES)
def test_bad_trees_are_refused_by_every_call(lib, change, status):
    want = getattr(lib, "ERR_" + status)
    for call in (_rope, _attn, _accept):
        assert call(lib, _tree(lib, **change)) == want
        assert call(lib, None) == lib.ERR_INVALID_ARG


@pytest.mark.parametrize("change,status", [
    (dict(qkv=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"),
    (dict(v=None), "INVALID_ARG"), (dict(hq=0), "INVALID_ARG"), (dict(base=0.0), "INVALID_ARG"),
    (dict(eps=-1.0), "INVALID_ARG"), (dict(d=96, ld=1024, ts=96), "UNSUPPORTED"), (dict(ld=64), "INVALID_ARG"),
    (dict(ts=32), "INVALID_ARG"), (dict(qkv=FAKE + 2), "ALIGNMENT"), (dict(ts=68), "ALIGNMENT"),
    (dict(ss=0), "INVALID_ARG"), (dict(ss=-64), "INVALID_ARG"),
])
def test_rope_append_tree_refusals(lib, change, status):
    assert _rope(lib, _tree(lib), **change) == getattr(lib, "ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
    (dict(hq=3, hkv=2), "INVALID_ARG"), (dict(hq=3), "UNSUPPORTED"), (dict(d=96, ts=96), "UNSUPPORTED"),
    (dict(split=128), "UNSUPPORTED"), (dict(ts=32), "INVALID_ARG"), (dict(ss=0), "INVALID_ARG"),
    (dict(k=FAKE + 8), "ALIGNMENT"), (dict(ws=FAKE + 4), "ALIGNMENT"), (dict(wsb=16), "WORKSPACE"),
])
def test_attn_tree_refusals(lib, change, status):
    assert _attn(lib, _tree(lib), **change) == getattr(lib, "ERR_" + status)


def test_attn_tree_bounds(lib):
    assert _attn(lib, _tree(lib, max_kv=0)) == lib.ERR_INVALID_ARG
    assert _attn(lib, _tree(lib, max_kv=256 * 65535 + 1), ss=64 * (256 * 65535 + 1)) == lib.ERR_UNSUPPORTED
    for nothing in (dict(B=0), dict(total_rows=0), dict(max_nodes=0)):
        assert _attn(lib, _tree(lib, **nothing)) == lib.OK
        assert _rope(lib, _tree(lib, **nothing)) == lib.OK
    L = lib.lib()
    assert L.kinv_attn_tree_workspace(2, 10, 8, 4, 2, 64, 0, 256) == 0
    need = L.kinv_attn_tree_workspace(2, 10, 8, 4, 2, 64, 512, 256)
    assert need > 0
    assert _attn(lib, _tree(lib), hq=4, hkv=2, ts=128, ss=128 * 512, wsb=need - 1) == lib.ERR_WORKSPACE


@pytest.mark.parametrize("change,status", [
    (dict(tok=None), "INVALID_ARG"), (dict(nxt=None), "INVALID_ARG"), (dict(n=None), "INVALID_ARG"),
    (dict(path=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"),
    (dict(layers=-1), "INVALID_ARG"), (dict(layers=65536), "UNSUPPORTED"), (dict(d=60), "UNSUPPORTED"),
    (dict(ts=32), "INVALID_ARG"), (dict(ss=0), "INVALID_ARG"), (dict(k=FAKE + 8), "ALIGNMENT"),
    (dict(ls=68), "ALIGNMENT"), (dict(ls=-64), "INVALID_ARG"), (dict(layers=2, ls=0), "INVALID_ARG"),
])
def test_tree_accept_refusals(lib, change, status):
    assert _accept(lib, _tree(lib), **change) == getattr(lib, "ERR_" + status)


def _score(lib, x=FAKE, dtype=1, ld=100, rows=2, V=100, ids=FAKE, n=1, lp=FAKE, ent=FAKE, k=2, ti=FAKE, tl=FAKE):
    return lib.lib().kinv_logprobs(x, dtype, ld, rows, V, ids, n, lp, ent, k, ti, tl, None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"), (dict(ld=99), "INVALID_ARG"),
    (dict(rows=-1), "INVALID_ARG"), (dict(V=0), "INVALID_ARG"), (dict(V=1048577, ld=1048577), "UNSUPPORTED"),
    (dict(n=-1), "INVALID_ARG"), (dict(ids=None), "INVALID_ARG"), (dict(lp=None), "INVALID_ARG"),
    (dict(k=-1), "INVALID_ARG"), (dict(k=33), "UNSUPPORTED"), (dict(k=5, V=4), "INVALID_ARG"),
    (dict(ti=None), "INVALID_ARG"), (dict(tl=None), "INVALID_ARG"), (dict(x=FAKE + 2), "ALIGNMENT"),
    (dict(x=FAKE + 1, dtype=0), "ALIGNMENT"),
])
def test_logprobs_refusals(lib, change, status):
    assert _score(lib, **change) == getattr(lib, "ERR_" + status)
    assert _score(lib, rows=0) == lib.OK


def test_python_wrappers_refuse_wrong_tensors(lib):
    i32 = dict(dtype=torch.int32)
    with pytest.raises(TypeError):
        lib.Tree(torch.zeros(1, dtype=torch.int64), torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(4, **i32), 4, 16)
    with pytest.raises(ValueError):  # not on a CUDA device
        lib.Tree(torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(4, **i32), 4, 16)
    with pytest.raises(TypeError):
        lib.logprobs(torch.zeros(2, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        lib.logprobs(torch.zeros(2, 8))


def test_accept_marked_refuses_other_marks(lib):
    call = lambda mark, **tree: lib.lib().kinv_tree_accept_marked(
        _tree(lib, **tree), FAKE, FAKE, FAKE, FAKE, 1, 64 * 1024, 64 * 512, 64, 1, 64, FAKE, FAKE, FAKE, mark, None)
    for mark in (8, -1, 1 << 30):
        assert call(mark) == lib.ERR_INVALID_ARG
    for change, status in BAD_TREES:
        assert call(7, **change) == getattr(lib, "ERR_" + status)
