"""CPU tests of the C ABI of the operators of several new tokens per stream
(include/convt_extend.h) and of their Python binding: exported symbols, struct sizes, refusals (all of
them before any device work), routes and parts, and tree_mask."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import convt_forward_amd as C
from convt_forward_amd import extend as X
from tests.test_decode_abi import BAD_CACHE, FAKE, desc, refs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "convt_extend.h")


def i64s(*v):
    return (ctypes.c_int64 * len(v))(*v)


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(convt_[a-z0-9_]+)\s*\(", src)))
    assert len(names) == 5, names
    for n in names:
        assert hasattr(X.lib(), n), n


def test_structs_are_the_headers(tmp_path):
    """Sizes and offsets of the binding's structs against a C compiler's, of the header itself."""
    structs = {"convt_append_problem": X.AppendProblem, "convt_window_problem": X.WindowProblem, "convt_tree_problem": X.TreeProblem,
               "convt_extend_info": X.ExtendInfo}
    lines = []
    for name, t in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in t._fields_]
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "convt_extend.h"\nint main(void) {' + "\n".join(lines) + "return 0; }\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I" + os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = [v for t in structs.values() for v in [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]]
    assert got == want


def append(tokens=3, rk=(128, 64), rv=(128, 64), qs=(256, 64), qos=(256, 64), heads=4, rotary=64, inter=0, reserved=0, q=FAKE, k=FAKE, v=FAKE,
           slots=FAKE, pos=FAKE, inv=FAKE, kc=FAKE, vc=FAKE, ks=None, vs=None, qo=FAKE, cache=()):
    rows = X.CacheRows(tokens, i64s(*rk), i64s(*rv))
    p = X.AppendProblem(desc(**dict(cache)), rows, i64s(*qs), i64s(*qos), heads, rotary, inter, reserved)
    return X.lib().convt_cache_append(ctypes.byref(p), q, k, v, slots, pos, inv, kc, vc, ks, vs, qo, None)


@pytest.mark.parametrize("kw", [dict(cache=kw) for kw in BAD_CACHE] + [
    dict(tokens=-1), dict(tokens=2 ** 31), dict(tokens=2 ** 29), dict(heads=-1), dict(rotary=63), dict(rotary=-2), dict(rotary=66), dict(inter=2),
    dict(inter=-1), dict(reserved=1), dict(rk=(-1, 64)), dict(rv=(128, -64)), dict(qs=(-1, 64)), dict(qos=(256, 0)), dict(qos=(0, 64)),
    dict(qs=(2 ** 41, 64)), dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(slots=None), dict(pos=None), dict(inv=None), dict(kc=None),
    dict(vc=None), dict(ks=FAKE), dict(vs=FAKE), dict(cache=dict(q=1)), dict(cache=dict(q=1), ks=FAKE), dict(heads=0), dict(heads=0, q=None),
    dict(heads=0, qo=None)])
def test_append_refuses(kw):
    assert append(**kw) == 1


def test_append_unsupported_and_empty():
    assert append(cache=dict(dim=513)) == 2 and append(cache=dict(dtype=3)) == 2
    assert X.lib().convt_cache_append(None, *[FAKE] * 11, None) == 1
    assert append(tokens=0, q=None, k=None, v=None, slots=None, pos=None, inv=None, qo=None) == 0


def window(max_length=64, tokens=2, qs=(256, 64), os_=(256, 64), width=4, stride=4, window=16, sinks=2, batch=2, heads=4, ragged=0, route=0, scale=0.125,
           reserved=0, **kw):
    return X.WindowProblem(desc(**kw), max_length, tokens, i64s(*qs), i64s(*os_), width, stride, window, sinks, batch, heads, ragged, route, scale, reserved)


def window_query(**kw):
    info = X.ExtendInfo()
    return X.lib().convt_window_query(*refs(window(**kw), info)), info


def tree(max_length=64, qs=(1024, 256, 64), os_=(1024, 256, 64), ts=(4, 1), width=4, stride=4, batch=2, drafts=4, heads=4, route=0, scale=0.125,
         reserved=0, **kw):
    return X.TreeProblem(desc(**kw), max_length, i64s(*qs), i64s(*os_), i64s(*ts), width, stride, batch, drafts, heads, route, scale, reserved)


def tree_query(**kw):
    info = X.ExtendInfo()
    return X.lib().convt_tree_query(*refs(tree(**kw), info)), info


SHARED = [dict(max_length=-1), dict(max_length=65), dict(width=-1), dict(stride=3), dict(heads=0), dict(heads=3), dict(route=3), dict(route=-1),
          dict(scale=float("nan")), dict(scale=float("inf")), dict(max_length=2 ** 31 - 1, width=2 ** 30, stride=2 ** 30)]
# `reserved` here is the problem's own
CACHES = [kw for kw in BAD_CACHE if "reserved" not in kw]


@pytest.mark.parametrize("kw", CACHES + SHARED + [
    dict(batch=-1, tokens=-1), dict(batch=1), dict(tokens=3), dict(tokens=-1, ragged=1), dict(ragged=2), dict(window=-1), dict(sinks=-1), dict(reserved=1),
    dict(qs=(-1, 64)), dict(os_=(256, 0))])
def test_window_refuses(kw):
    assert window_query(**kw)[0] == 1


@pytest.mark.parametrize("kw", CACHES + SHARED + [
    dict(batch=-1), dict(drafts=0), dict(drafts=-1), dict(qs=(1024, -1, 64)), dict(os_=(1024, 256, 0)), dict(os_=(0, 256, 64)), dict(ts=(-1, 1)),
    dict(ts=(4, 2 ** 41)), dict(reserved=1)])
def test_tree_refuses(kw):
    assert tree_query(**kw)[0] == 1


def test_unsupported_requests():
    for query in (window_query, tree_query):
        assert query(dim=513)[0] == 2 and query(dtype=4)[0] == 2
        assert query(dtype=0, route=2)[0] == 2 and query(page=8, route=2, max_length=8)[0] == 2 and query(dim=40, route=2)[0] == 2
    assert window_query(batch=2 ** 22, tokens=2 ** 22)[0] == 2 and window_query(ragged=1, tokens=2 ** 40)[0] == 2
    assert tree_query(drafts=1025)[0] == 2 and tree_query(batch=2 ** 20, drafts=4)[0] == 2


def test_pointers_are_checked():
    def call(p, q=FAKE, kc=FAKE, vc=FAKE, ks=None, vs=None, pt=FAKE, ln=FAKE, more=None, out=FAKE, ws=None):
        f = X.lib().convt_window_attend if isinstance(p, X.WindowProblem) else X.lib().convt_tree_attend
        return f(ctypes.byref(p), q, kc, vc, ks, vs, pt, ln, more, out, None, ws, None)
    for p, more in ((window(), None), (window(ragged=1), FAKE), (tree(), FAKE)):
        for kw in [dict(q=None), dict(kc=None), dict(vc=None), dict(ks=FAKE), dict(pt=None), dict(ln=None), dict(out=None)]:
            assert call(p, more=more, **kw) == 1, kw
    assert call(window(), more=FAKE) == 1 and call(window(ragged=1)) == 1 and call(tree()) == 1 and call(tree(), more=FAKE + 4) == 1
    assert call(window(q=1)) == 1 and call(tree(q=1), more=FAKE, ks=FAKE) == 1
    far = dict(max_length=2 ** 20, width=2 ** 16, stride=2 ** 16)
    assert window_query(window=0, **far)[1].workspace_bytes > 0 and tree_query(**far)[1].workspace_bytes > 0
    for ws in (None, FAKE + 8):
        assert call(window(window=0, **far), ws=ws) == 1 and call(tree(**far), more=FAKE, ws=ws) == 1
    assert call(window(batch=0, tokens=0), q=None, pt=None, ln=None, out=None) == 0
    assert call(window(tokens=0, ragged=1), q=None, pt=None, ln=None, out=None) == 0
    assert call(tree(batch=0), q=None, pt=None, ln=None, out=None) == 0
    assert X.lib().convt_window_query(None, None) == 1 and X.lib().convt_tree_query(None, None) == 1


@pytest.mark.parametrize("dim,dtype", [(64, 1), (128, 1), (256, 2), (33, 0)])
@pytest.mark.parametrize("length", [0, 1, 63, 64, 65, 513, 4096, 100000, 2 ** 30, 2 ** 31 - 4097])
@pytest.mark.parametrize("batch", [1, 7, 512])
def test_parts_cover_what_is_seen(length, batch, dim, dtype):
    far = dict(width=2 ** 27, stride=2 ** 27, batch=batch, dim=dim, dtype=dtype, max_length=length)
    asked = [(window_query(tokens=batch, window=0, **far), length, batch), (tree_query(drafts=9, **far), length, 9 * batch),
             (window_query(tokens=40 * batch, ragged=1, window=0, **far), length, 40 * batch)]
    for w, k in ((1, 0), (100, 70), (2 ** 40, 2 ** 40), (70, 2 ** 62)):
        asked.append((window_query(tokens=batch, window=w, sinks=k, **far), min(length, w + k), batch))
    for (st, i), sees, rows in asked:
        assert st == 0
        assert 1 <= i.chunks <= 32768 and i.chunks * i.chunk_tokens >= sees and i.chunk_tokens % 64 == 0
        assert i.workspace_bytes == (0 if i.chunks == 1 else rows * 4 * (i.chunks * (dim + 2) + 1) * 4)


def test_python_refuses_host_tensors_and_wrong_names():
    with pytest.raises(ValueError, match="device tensor"):
        C.KVCache(torch.zeros(1, 1, 16, 8), torch.zeros(1, 1, 16, 8))
    with pytest.raises(AttributeError):
        C.no_such_attention
    for name in ("cache_append", "window_attention", "tree_attention", "tree_mask", "window_plan", "tree_plan", "EXTEND_ROUTES"):
        assert hasattr(C, name)


def ancestors(parents):
    rows = []
    for i in range(len(parents)):
        bits, j = 0, i
        while j >= 0:
            bits |= 1 << j
            j = parents[j]
        rows.append(bits)
    return rows


@pytest.mark.parametrize("drafts", [1, 2, 3, 25, 63, 64, 65, 130, 1024])
def test_tree_mask(drafts):
    g = torch.Generator().manual_seed(drafts)
    parents = (torch.rand(2, 3, drafts, generator=g) * (torch.arange(drafts) + 1)).long() - 1
    parents[0, 0] = torch.arange(-1, drafts - 1)  # a chain
    parents[0, 1] = -1
    # any order: the drafts of one tree shuffled
    order = torch.randperm(drafts, generator=g)
    shuffled = torch.empty(drafts, dtype=torch.long)
    shuffled[order] = torch.where(parents[1, 0] >= 0, order[parents[1, 0].clamp(min=0)], -1)
    parents[1, 1] = shuffled
    got = C.tree_mask(parents.to(torch.int32))
    assert got.dtype == torch.int64 and got.shape == (2, 3, drafts, (drafts + 63) // 64)
    for a in range(2):
        for b in range(3):
            rows = [sum((w & (2 ** 64 - 1)) << 64 * i for i, w in enumerate(r)) for r in got[a, b].tolist()]
            assert rows == ancestors(parents[a, b].tolist()), (a, b)
