"""CPU tests of the decoding-step operators' C ABI (include/convt_decode.h) and Python
binding: exported symbols, refusals (all of them before any device work), the choice of
route and split, and the helpers that are plain torch."""
import ctypes
import os
import re

import pytest
import torch

import convt_forward_amd as C
from convt_forward_amd import decode as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # an aligned address that is never followed: every call here is refused first


def refs(*s):
    return [ctypes.byref(v) for v in s]


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "convt_decode.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(convt_[a-z0-9_]+)\s*\(", src)))
    assert len(names) == 7, names
    for n in names:
        assert hasattr(D.lib(), n), n


def norm(rows=4, width=64, xs=64, rs=64, ys=64, ros=64, dtype=1, res=1, q=0, eps=1e-6, x=FAKE, w=FAKE, r=FAKE, y=FAKE,
         s=None, ro=FAKE):
    p = D.NormProblem(rows, width, xs, rs, ys, ros, dtype, res, q, eps)
    return D.lib().convt_rms_norm(ctypes.byref(p), x, w, r, y, s, ro, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(width=0), dict(width=2 ** 24 + 1), dict(xs=63), dict(rs=63), dict(ys=63), dict(ros=63),
    dict(xs=-64), dict(xs=2 ** 41), dict(dtype=-1), dict(dtype=99), dict(res=2), dict(q=2), dict(q=-1), dict(eps=-1e-6),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None), dict(y=None), dict(r=None),
    dict(ro=None), dict(res=0), dict(res=0, r=None), dict(q=1), dict(s=FAKE)])
def test_norm_refuses(kw):
    assert norm(**kw) == 1


def test_norm_unsupported_types_and_empty():
    assert [norm(dtype=d) for d in (3, 4, 5)] == [2, 2, 2]
    assert D.lib().convt_rms_norm(None, FAKE, FAKE, FAKE, FAKE, None, FAKE, None) == 1
    # no rows: nothing to do, whatever the pointers
    assert norm(rows=0, x=None, w=None, r=None, y=None, ro=None) == 0


def desc(pages=8, ks=(2048, 1024, 64), vs=(2048, 1024, 64), heads=2, page=16, dim=64, dtype=1, q=0, reserved=0):
    return D.CacheDesc(pages, (ctypes.c_int64 * 3)(*ks), (ctypes.c_int64 * 3)(*vs), heads, page, dim, dtype, q, reserved)


BAD_CACHE = [dict(pages=-1), dict(heads=0), dict(page=0), dict(dim=0), dict(dtype=42), dict(q=2), dict(reserved=1),
             dict(ks=(2048, 0, 64)), dict(vs=(-1, 1024, 64)), dict(ks=(2048, 1024, 2 ** 41)),
             dict(pages=2 ** 27, page=16), dict(pages=2 ** 62)]


def move(which, c, tokens=3, k=FAKE, v=FAKE, slots=FAKE, kc=FAKE, vc=FAKE, ks=None, vs=None, rk=(128, 64), rv=(128, 64)):
    r = D.CacheRows(tokens, (ctypes.c_int64 * 2)(*rk), (ctypes.c_int64 * 2)(*rv))
    if which == "write":
        return D.lib().convt_cache_write(*refs(c, r), k, v, slots, kc, vc, ks, vs, None)
    return D.lib().convt_cache_read(*refs(c, r), kc, vc, ks, vs, slots, k, v, None)


@pytest.mark.parametrize("which", ["write", "read"])
def test_cache_refuses(which):
    for kw in BAD_CACHE:
        assert move(which, desc(**kw)) == 1, kw
    for kw in [dict(tokens=-1), dict(tokens=2 ** 31), dict(tokens=2 ** 30), dict(k=None), dict(v=None),
               dict(slots=None), dict(kc=None), dict(vc=None), dict(ks=FAKE), dict(vs=FAKE), dict(rk=(-1, 64)),
               dict(rv=(128, -64))]:
        assert move(which, desc(), **kw) == 1, kw
    for kw in [dict(), dict(ks=FAKE), dict(vs=FAKE)]:
        assert move(which, desc(q=1), **kw) == 1, kw
    if which == "read":  # written rows may not coincide
        assert move(which, desc(), rk=(0, 64)) == 1 and move(which, desc(), rv=(128, 0)) == 1
    assert move(which, desc(dim=513)) == 2
    assert move(which, desc(dtype=3)) == 2
    assert move(which, desc(), tokens=0, k=None, v=None, slots=None) == 0
    # a cache without pages takes no token
    if which == "write":
        assert move(which, desc(pages=0), kc=None, vc=None) == 0


def problem(max_length=64, qs=(256, 64), os_=(256, 64), width=4, stride=4, batch=2, heads=4, route=0, scale=0.125, **kw):
    return D.AttendProblem(desc(**kw), max_length, (ctypes.c_int64 * 2)(*qs), (ctypes.c_int64 * 2)(*os_), width, stride,
                           batch, heads, route, scale)


def query(**kw):
    info = D.AttendInfo()
    return D.lib().convt_attend_query(*refs(problem(**kw), info)), info


@pytest.mark.parametrize("kw", BAD_CACHE + [
    dict(max_length=-1), dict(max_length=65), dict(qs=(-1, 64)), dict(os_=(256, 0)), dict(width=-1), dict(stride=3),
    dict(batch=-1), dict(heads=0), dict(heads=3), dict(route=3), dict(route=-1), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(max_length=2 ** 31 - 1, width=2 ** 30, stride=2 ** 30)])
def test_attend_refuses(kw):
    assert query(**kw)[0] == 1


def test_attend_refuses_pointers():
    def call(p, q=FAKE, kc=FAKE, vc=FAKE, ks=None, vs=None, pt=FAKE, ln=FAKE, out=FAKE, ws=None):
        return D.lib().convt_attend(ctypes.byref(p), q, kc, vc, ks, vs, pt, ln, out, None, ws, None)
    for kw in [dict(q=None), dict(kc=None), dict(vc=None), dict(ks=FAKE), dict(pt=None), dict(ln=None), dict(out=None)]:
        assert call(problem(), **kw) == 1, kw
    assert call(problem(q=1)) == 1 and call(problem(q=1), ks=FAKE) == 1
    long = problem(max_length=16384, width=1024, stride=1024)
    assert query(max_length=16384, width=1024, stride=1024)[1].workspace_bytes > 0
    assert call(long) == 1 and call(long, ws=FAKE + 8) == 1
    assert call(problem(batch=0), q=None, pt=None, ln=None, out=None) == 0
    assert D.lib().convt_attend_query(None, None) == 1


def test_attend_unsupported():
    assert query(dim=513)[0] == 2
    assert query(batch=2 ** 22, heads=4)[0] == 2
    assert query(dtype=4)[0] == 2


@pytest.mark.parametrize("length", [0, 1, 255, 256, 257, 4096, 100000, 2 ** 30])
@pytest.mark.parametrize("batch", [1, 7, 512])
def test_attend_parts_cover_the_length(length, batch):
    st, i = query(max_length=length, width=2 ** 27, stride=2 ** 27, batch=batch)
    assert st == 0
    assert 1 <= i.chunks <= 32768 and i.chunks * i.chunk_tokens >= length and (i.chunks - 1) * i.chunk_tokens <= length
    assert i.workspace_bytes == (0 if i.chunks == 1 else batch * 4 * i.chunks * (64 + 2) * 4)


def q4(rows=3, n=5, k=64, group=32, xs=64, ys=5, dtype=1, q=0, route=0, reserved=0, x=FAKE, s=None, w=FAKE, sc=FAKE, y=FAKE):
    p = D.Q4Problem(rows, n, k, group, xs, ys, dtype, q, route, reserved)
    return D.lib().convt_q4_matvec(ctypes.byref(p), x, s, w, sc, y, None)


def test_q4_refuses():
    for kw in [dict(rows=-1), dict(n=-1), dict(k=-1), dict(k=2 ** 31), dict(rows=2 ** 31), dict(n=2 ** 31), dict(group=0),
               dict(group=4), dict(group=12), dict(group=-32), dict(k=48), dict(xs=63), dict(ys=4), dict(dtype=77),
               dict(q=2), dict(q=1), dict(route=3), dict(route=-1), dict(reserved=1), dict(x=None), dict(w=None),
               dict(sc=None), dict(y=None), dict(s=FAKE)]:
        assert q4(**kw) == 1, kw
    assert q4(dtype=3) == 2 and q4(n=2 ** 30, ys=2 ** 30) == 2
    assert q4(rows=0, x=None, w=None, sc=None, y=None) == 0 and q4(n=0, y=None) == 0
    assert D.lib().convt_q4_query(None, None) == 1


def test_python_refuses_host_tensors_and_wrong_shapes():
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="device tensor"):
        C.rms_norm(x, w)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        C.rms_norm(x.to(torch.int32), w)
    with pytest.raises(ValueError, match="device tensor"):
        C.KVCache(torch.zeros(1, 1, 16, 8), torch.zeros(1, 1, 16, 8))
    with pytest.raises(ValueError, match="go together"):
        C.KVCache(torch.zeros(1, 1, 16, 8), torch.zeros(1, 1, 16, 8), torch.zeros(1, 1, 16))
    with pytest.raises(ValueError, match="n_pages"):
        C.KVCache(x, x)
    with pytest.raises(ValueError, match="device tensor"):
        C.q4_matvec(x, torch.zeros(3, 4, dtype=torch.uint8), torch.zeros(3, 1))
    with pytest.raises(AttributeError):
        C.no_such_operator


def test_row_spacing():
    t = torch.zeros(4, 6, 8)
    assert D._rows(t, "t") == (24, 8)
    assert D._rows(t[:, :, :5], "t") == (24, 8)
    assert D._rows(t[:1, ::2], "t") == (3, 16)
    assert D._rows(torch.zeros(8), "t")[0] == 1
    with pytest.raises(ValueError, match="evenly spaced"):
        D._rows(t[:, :3], "t")
    with pytest.raises(ValueError, match="contiguous"):
        D._rows(t.transpose(1, 2), "t")


def test_q4_quantise_round_trip():
    g = torch.Generator().manual_seed(1)
    w = torch.randn(5, 64, generator=g)
    w[2, :32] = 0
    codes, scales = C.q4_quantise(w, 32)
    assert codes.dtype == torch.uint8 and codes.shape == (5, 32) and scales.shape == (5, 2)
    back = torch.stack([codes & 15, codes >> 4], -1).reshape(5, 64).float() - 8
    back = back * scales.repeat_interleave(32, 1)
    # half a step, and the step's own rounding over 7 of them
    assert ((back - w).abs() <= scales.repeat_interleave(32, 1) * (0.5 + 8 * 2.0 ** -24)).all()
    assert (back[2, :32] == 0).all()
    for group in (0, 4, 12, 48):
        with pytest.raises(ValueError):
            C.q4_quantise(w, group)


def test_cache_slots():
    table = torch.tensor([[3, 0], [7, 5]], dtype=torch.int32)
    got = C.cache_slots(table, torch.tensor([0, 1, 1]), torch.tensor([17, 0, 31]), 16)
    assert got.dtype == torch.int64 and got.tolist() == [0 * 16 + 1, 7 * 16, 5 * 16 + 15]
