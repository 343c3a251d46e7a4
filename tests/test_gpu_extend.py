"""GPU tests of the operators of several new tokens per stream against their plain 64-bit forms
(tests/extend_util.py): sizes that end inside a piece, a tile or a page, strides, rows that see
nothing, NaN and infinities where they must not be read, pages and slots outside the cache,
parts of the length axis, streams and graph replays."""
import math

import pytest
import torch

import convt_forward_amd as C
from tests.decode_util import E4M3, TYPES, U, quantised_bound, rounding, within
from tests.extend_util import (DEV, Streams, attend64, p_step, rand, rotate64, rotated_bound, row_bound, tree_seen, window_seen)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- cache_append


def freqs(half, base=10000.0):
    return base ** (-torch.arange(half, dtype=torch.float32) / max(1, half))


def check_append(dt, quantised, dim, rotary, interleaved, tokens, heads=3, kv=2, page=16, positions=None, slots=None, in_place=False):
    print(f"append {dt} q8 {quantised} dim {dim} rotary {rotary} inter {interleaved} tokens {tokens}", flush=True)
    t = TYPES[dt]
    pages = -(-tokens // page) + 2
    cache = C.KVCache.new(pages, kv, page, dim, dtype=t, quantised=quantised)
    g = torch.Generator().manual_seed(tokens + dim)
    if slots is None:
        slots = torch.randperm(pages * page, generator=g)[:tokens]
    if positions is None:
        positions = torch.randint(0, 200000, (tokens,), generator=g)
    qkv = rand(tokens, heads + 2 * kv, dim, seed=3).to(t)
    inv = freqs(rotary // 2)
    dev = qkv.to(DEV)
    q, k, v = dev.split([heads, kv, kv], 1)
    kept_k, kept_v = cache.k.clone(), cache.v.clone()
    got = C.cache_append(cache, k, v, slots.to(DEV), positions.to(DEV), inv.to(DEV), q=q, interleaved=interleaved, q_out=q if in_place else None)
    torch.cuda.synchronize()
    hq, hk, hv = qkv.double().split([heads, kv, kv], 1)
    want, mag = rotate64(hq, positions, inv, interleaved)
    within(got, want, rounding(t, want) * (1 + 2.0 ** -10) + rotated_bound(mag), "q")
    assert torch.equal(dev[:, heads:].cpu(), qkv[:, heads:])
    inside = (slots >= 0) & (slots < pages * page)
    at = slots[inside]
    for name, x in (("k", rotate64(hk, positions, inv, interleaved)), ("v", (hv, torch.zeros_like(hv)))):
        want, off = x[0][inside], rotated_bound(x[1][inside])
        cells = getattr(cache, name).cpu()
        got = cells.transpose(1, 2).reshape(pages * page, kv, dim)
        if quantised:
            scale = getattr(cache, name + "_scale").cpu().transpose(1, 2).reshape(pages * page, kv)[at].double()
            s64 = (want.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
            within(scale, s64, s64 * 2 * U + off.amax(-1) / 448, name + " scale")
            within(got[at].double() * scale.unsqueeze(-1), want, quantised_bound(want, s64) + 2 * off + off.amax(-1, keepdim=True) * 2.0 ** -3, name)
        else:
            within(got[at], want, rounding(t, want) * (1 + 2.0 ** -10) + off, name)
        # other places are as they were
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[at] = False
        old = (kept_k if name == "k" else kept_v).cpu().transpose(1, 2).reshape(pages * page, kv, dim)
        assert torch.equal(got[rest].view(torch.uint8 if quantised else t), old[rest].view(torch.uint8 if quantised else t))


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dim,rotary", [(2, 2), (8, 8), (20, 12), (64, 64), (64, 32), (64, 24), (80, 80), (96, 64), (97, 96), (128, 128),
                                        (256, 256), (512, 510), (512, 512), (33, 0)])
def test_append_dims(dt, quantised, dim, rotary):
    for interleaved in (False, True):
        check_append(dt, quantised, dim, rotary, interleaved, 5)


@pytest.mark.parametrize("tokens", [0, 1, 3, 63, 4095, 4096, 4099])
@pytest.mark.parametrize("quantised", [False, True])
def test_append_tokens(tokens, quantised):
    check_append("bf16", quantised, 64, 64, False, tokens, heads=5, kv=1)
    check_append("f16", quantised, 48, 48, True, tokens, heads=1, kv=3, in_place=True)


def test_append_in_place_and_odd_sizes():
    check_append("f32", False, 72, 36, False, 130, heads=7, kv=2, page=5, in_place=True)
    check_append("bf16", True, 128, 128, False, 130, heads=33, kv=8, page=3, in_place=True)


@pytest.mark.parametrize("first", [0, -5, 131072, 10 ** 6, 2 ** 31, 2 ** 40, -2 ** 40])
def test_append_positions_keep_their_angles(first):
    # in float32 the largest of these would be off by whole turns; the product of two factors
    # rounded to 53 bits is off by 2^-53 of itself
    tokens, half = 40, 16
    positions = first + torch.arange(tokens) * 3
    inv = freqs(half, 500000.0)
    q = rand(tokens, 2, 2 * half)
    cache = C.KVCache.new(4, 1, 16, 2 * half, dtype=torch.float32)
    k = rand(tokens, 1, 2 * half, seed=5)
    got = C.cache_append(cache, k.to(DEV), k.to(DEV), torch.arange(tokens, device=DEV), positions.to(DEV), inv.to(DEV), q=q.to(DEV))
    exact = [[(int(p) * int(float(f) * 2 ** 60)) for f in inv] for p in positions]  # float32 values are whole multiples of 2^-60 here
    # 2 pi to 200 bits by whole numbers: the angle modulo a turn, exactly, before it becomes a float
    turn = 10096689509235987743946820282484873672429286842977325943070736  # floor(2 pi 2^200)
    assert abs(turn / 2 ** 200 - 2 * math.pi) < 1e-15
    angle = torch.tensor([[((e << 140) % turn) / 2 ** 200 for e in row] for row in exact], dtype=torch.float64)
    a, b = q.double()[..., :half], q.double()[..., half:]
    c, s = angle.cos().unsqueeze(1), angle.sin().unsqueeze(1)
    want = torch.cat([a * c - b * s, a * s + b * c], -1)
    mag = (a.abs() + b.abs()).repeat(1, 1, 2)
    far = (abs(first) + 200) * 2.0 ** -52
    within(got, want, rounding(torch.float32, want) + rotated_bound(mag, far), f"first {first}")


def test_append_slots_outside_and_padding():
    # three pages of 16
    slots = torch.tensor([5, -1, 3 * 16 - 1, 3 * 16, -2 ** 40, 2 ** 40, 0])
    for quantised in (False, True):
        check_append("bf16", quantised, 64, 64, False, 7, page=16, slots=slots)


def test_append_without_rotation_is_cache_write():
    for quantised in (False, True):
        a, b = (C.KVCache.new(8, 2, 16, 96, quantised=quantised) for _ in range(2))
        k, v = rand(100, 2, 96).bfloat16().to(DEV), rand(100, 2, 96, seed=1).bfloat16().to(DEV)
        slots = torch.randperm(128, generator=torch.Generator().manual_seed(0))[:100].to(DEV)
        none = torch.zeros(0, device=DEV)
        assert C.cache_append(a, k, v, slots, torch.zeros(100, dtype=torch.int64, device=DEV), none) is None
        C.cache_write(b, k, v, slots)
        for x, y in ((a.k, b.k), (a.v, b.v)) + (((a.k_scale, b.k_scale), (a.v_scale, b.v_scale)) if quantised else ()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_special_values():
    k = rand(4, 1, 32)
    k[0] = 0
    k[1, 0, 3] = math.nan
    k[2, 0, 5] = math.inf
    cache = C.KVCache.new(1, 1, 16, 32, quantised=True)
    pos = torch.arange(4)
    C.cache_append(cache, k.to(DEV), k.to(DEV), pos.to(DEV), pos.to(DEV), freqs(16).to(DEV))
    back, _ = C.cache_read(cache, pos.to(DEV), dtype=torch.float32)
    back = back.cpu()
    assert (back[0] == 0).all() and back[1].isnan().all() and back[2].isnan().all() and back[3].isfinite().all()
    # a frequency that is not a number turns only its own pair to NaN
    inv = freqs(16)
    inv[2] = math.nan
    cache = C.KVCache.new(1, 1, 16, 32, dtype=torch.float32)
    q = C.cache_append(cache, k.to(DEV), k.to(DEV), pos.to(DEV), pos.to(DEV), inv.to(DEV), q=k.to(DEV)).cpu()
    bad = q[3, 0].isnan().nonzero().flatten().tolist()
    assert bad == [2, 18]


def test_append_strided_cache_and_rows():
    t = torch.float16
    for quantised in (False, True):
        ref = C.KVCache.new(6, 2, 16, 64, dtype=t, quantised=quantised)
        k = torch.zeros(6, 16, 2, 64, dtype=torch.uint8 if quantised else t, device=DEV)
        v = torch.zeros_like(k)
        if quantised:
            k, v = k.view(E4M3), v.view(E4M3)
        other = C.KVCache(k.transpose(1, 2), v.transpose(1, 2), *((torch.zeros(6, 2, 16, device=DEV) for _ in range(2)) if quantised else ()))
        wide = rand(50, 9, 70).to(t).to(DEV)
        kk, vv, q = wide[:, 1:3, 3:67], wide[:, 4:6, 3:67], wide[:, 6:9, 5:69]
        slots, pos = torch.arange(50, device=DEV) + 7, torch.arange(50, device=DEV)
        out = torch.full((50, 4, 66), 7.0, dtype=t, device=DEV)
        a = C.cache_append(ref, kk.contiguous(), vv.contiguous(), slots, pos, freqs(32).to(DEV), q=q.contiguous())
        b = C.cache_append(other, kk, vv, slots, pos, freqs(32).to(DEV), q=q, q_out=out[:, :3, 1:65])
        assert torch.equal(a, b) and (out[:, 3] == 7).all() and (out[:, :, 0] == 7).all() and (out[:, :, 65] == 7).all()
        assert torch.equal(ref.k.view(torch.uint8), other.k.contiguous().view(torch.uint8))
        assert torch.equal(ref.v.view(torch.uint8), other.v.contiguous().view(torch.uint8))
        if quantised:
            assert torch.equal(ref.k_scale, other.k_scale) and torch.equal(ref.v_scale, other.v_scale)


# ---------------------------------------------------------------- window_attention


def check_window(streams, lengths, news, heads, window, sinks, route="auto", scale=None, spare=0, lse=True, seed=0, q=None, max_length=None):
    """lengths and news per stream; the rows behind the last stream keep what they hold."""
    s, dt = streams, streams.dt
    t = TYPES[dt]
    rows = sum(news) + spare
    q = rand(rows, heads, s.dim, seed=seed + 11, scale=2).to(t) if q is None else q
    starts = torch.tensor([0] + list(news)).cumsum(0).to(torch.int32)
    single = spare == 0 and all(n == 1 for n in news)
    out = torch.full((rows, heads, s.dim), 7.0, dtype=t, device=DEV)
    lse_t = torch.full((rows, heads), 7.0, device=DEV)
    real = s.dim ** -0.5 if scale is None else scale
    plan = C.window_plan(s.cache, q.to(DEV), s.table.to(DEV), not single, window, sinks, scale, max_length, out, route)[1]
    print(f"window {dt} q8 {s.cache.quantised} dim {s.dim} page {s.page} heads {heads} lengths {lengths} new {news} window {window} sinks {sinks} "
          f"route {plan.route} chunks {plan.chunks}", flush=True)
    got, got_lse = C.window_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV),
                                      starts=None if single else starts.to(DEV), window=window, sinks=sinks, scale=scale, max_length=max_length,
                                      out=out, lse=lse_t, route=route)
    torch.cuda.synchronize()
    assert got is out
    k, v, valid = s.tokens64("k"), s.tokens64("v"), s.page_seen()
    step = p_step(dt, s.cache.quantised, "direct" if plan.route == 1 else "mfma")
    for b, n in enumerate(news):
        if n == 0:
            continue
        length = max(0, min(lengths[b], s.room if max_length is None else max_length))
        seen = window_seen(length, n, s.room, window, sinks) & valid[b]
        at = slice(int(starts[b]), int(starts[b + 1]))
        want, want_lse, mag, top = attend64(q[at], k[b], v[b], seen, real)
        most = int(seen.sum(1).max())
        within(got[at], want, row_bound(want, mag, top, s.dim, most, dt, step, s.cache.quantised), f"stream {b}")
        within(got_lse[at], want_lse, (2 * (s.dim + 12) * U * top + (most + 64) * U + 2.0 ** -17 + want_lse.abs().nan_to_num(0, 0, 0) * 4 * U), f"lse {b}")
    assert (got[sum(news):] == 7).all() and (got_lse[sum(news):] == 7).all()
    return got


ROUTES = ["direct", "auto"]


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dt,quantised", [("bf16", False), ("bf16", True), ("f16", False), ("f16", True), ("f32", False), ("f32", True)])
@pytest.mark.parametrize("dim,page,heads,kv", [(64, 16, 4, 2), (128, 16, 8, 2), (96, 32, 5, 1), (80, 16, 6, 3), (256, 16, 4, 1), (16, 16, 2, 2),
                                               (208, 48, 3, 1), (176, 16, 2, 2), (33, 7, 3, 1), (320, 16, 2, 1)])
def test_window_types_and_dims(route, dt, quantised, dim, page, heads, kv):
    s = Streams(3, 150, kv, dim, page, dt, quantised)
    check_window(s, [150, 67, 13], [40, 67, 1], heads, 33, 3, route)
    check_window(s, [150, 67, 13], [1, 1, 1], heads, 33, 3, route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (1, 1), (2, 64), (16, 4), (63, 65), (64, 0), (65, 200), (100, 17), (128, 128), (1000, 5)])
@pytest.mark.parametrize("quantised", [False, True])
def test_window_masks(route, window, sinks, quantised):
    s = Streams(2, 333, 1, 64, 16, "bf16", quantised, seed=4)
    check_window(s, [333, 190], [333, 65], 4, window, sinks, route)
    check_window(s, [333, 129], [17, 1], 4, window, sinks, route)
    check_window(s, [330, 64], [1, 1], 4, window, sinks, route)


@pytest.mark.parametrize("route", ROUTES)
def test_window_ragged_rows_empty_streams_and_rows_behind(route):
    s = Streams(6, 100, 2, 64, 16, "f16", False, seed=5)
    # streams without rows, without tokens, with more rows than tokens
    check_window(s, [100, 0, 50, 3, 0, 99], [5, 0, 0, 7, 2, 40], 4, 20, 2, route, spare=9)
    check_window(s, [0] * 6, [1] * 6, 4, 20, 2, route)
    check_window(s, [0] * 6, [0] * 6, 4, 20, 2, route, spare=5)
    check_window(s, [-3, 100, 1, 2, 17, 16], [1] * 6, 4, None, 0, route)
    check_window(s, [100] * 6, [0, 0, 0, 0, 0, 1], 4, 7, 0, route, spare=2)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("share", [1, 2, 3, 5, 7, 16, 17, 33, 40, 130])
def test_window_shared_heads(route, share):
    s = Streams(2, 90, 2, 64, 16, "bf16", False, seed=share)
    check_window(s, [90, 40], [33, 6], 2 * share, 30, 2, route)
    check_window(s, [90, 40], [1, 1], 2 * share, 30, 2, route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("quantised", [False, True])
def test_window_parts_are_joined(route, quantised):
    s = Streams(2, 6000, 1, 64, 16, "bf16", quantised, seed=6)
    assert check_window(s, [5999, 4100], [1, 1], 2, None, 0, route) is not None
    check_window(s, [5999, 33], [3, 2], 2, None, 0, route, spare=1)
    check_window(s, [5999, 4100], [9, 1], 2, 5000, 70, route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_window_bad_values_where_a_row_does_not_see(route, quantised, dt):
    """Tokens that some rows see and others do not hold NaN or infinities: only the former change."""
    for value in (math.nan, math.inf, -math.inf):
        if quantised and not math.isnan(value):
            continue
        s = Streams(2, 200, 1, 64, 16, dt, quantised, seed=7)
        for name in "kv":
            for b, t in ((0, 150), (0, 5), (1, 199)):
                s.set(name, b, t, value)
        q = rand(60 + 199, 2, 64, seed=3, scale=2).to(TYPES[dt])
        starts = torch.tensor([0, 60, 259], dtype=torch.int32, device=DEV)
        lengths = torch.tensor([180, 199], dtype=torch.int32, device=DEV)
        got = C.window_attention(q.to(DEV), s.cache, s.table.to(DEV), lengths, starts=starts, window=25, sinks=3, route=route).cpu()
        # stream 0: positions 120 .. 179 see 150 from 150 to 174, and never 5; stream 1 sees 5 tokens behind none
        bad = torch.zeros(259, dtype=torch.bool)
        bad[30:55] = True
        assert got[~bad].isfinite().all(), value
        assert got[bad].isnan().all(), value
        # values alone: what is seen is what the formula gives
        s = Streams(1, 200, 1, 64, 16, dt, quantised, seed=8)
        s.set("v", 0, 100, value)
        check_window(s, [180], [100], 2, 25, 3, route)
        check_window(s, [110], [3], 2, 25, 3, route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("quantised", [False, True])
def test_window_pages_outside_the_cache_are_left_out(route, quantised):
    s = Streams(2, 200, 2, 64, 16, "bf16", quantised, seed=9)
    s.table[0, 3], s.table[1, 0], s.table[0, 12], s.table[1, 5] = -1, 10 ** 6, -2 ** 31, 2 ** 31 - 1
    check_window(s, [190, 150], [70, 150], 4, 60, 20, route)
    check_window(s, [190, 90], [1, 1], 4, None, 0, route)
    s.table[:] = -1
    check_window(s, [190, 150], [70, 2], 4, 60, 20, route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 1e-30, 3e3])
def test_window_scales(route, scale):
    s = Streams(1, 150, 1, 64, 16, "f16", False, seed=10)
    if abs(scale) > 100:
        # few keys count: scores that differ by less than their own roundings are kept out
        s = Streams(1, 150, 1, 64, 16, "f16", False, seed=10, scale=1e-3)
    check_window(s, [150], [20], 2, 50, 2, route, scale=scale)
    check_window(s, [150], [1], 2, 50, 2, route, scale=scale)


@pytest.mark.parametrize("route", ROUTES)
def test_window_strides_layouts_and_max_length(route):
    for quantised in (False, True):
        s = Streams(2, 130, 2, 64, 16, "bf16", quantised, seed=11, layout="token")
        check_window(s, [130, 77], [30, 9], 4, 50, 2, route)
        check_window(s, [130, 77], [30, 9], 4, 50, 2, route, max_length=100)
        check_window(s, [130, 77], [1, 1], 4, 50, 2, route, max_length=0)
        q = rand(39, 4, 64, seed=2).bfloat16().to(DEV)
        starts, lengths = torch.tensor([0, 30, 39], dtype=torch.int32, device=DEV), torch.tensor([130, 77], dtype=torch.int32, device=DEV)
        table = s.table.to(DEV)
        want = C.window_attention(q, s.cache, table, lengths, starts=starts, window=50, sinks=2, route=route)
        wide = torch.full((39, 6, 80), 5.0, dtype=torch.bfloat16, device=DEV)
        qw = torch.zeros(39, 7, 72, dtype=torch.bfloat16, device=DEV)
        qw[:, 1:5, 8:72] = q
        got = C.window_attention(qw[:, 1:5, 8:72], s.cache, torch.cat([table, table], 1)[:, :table.shape[1]], lengths, starts=starts, window=50, sinks=2,
                                 out=wide[:, 1:5, 9:73], route=route)
        assert torch.equal(got, want) and (wide[:, 0] == 5).all() and (wide[:, :, :9] == 5).all() and (wide[:, :, 73:] == 5).all()
        # a query that starts at any element
        qo = torch.zeros(39, 4, 71, dtype=torch.bfloat16, device=DEV)
        qo[:, :, 3:67] = q
        got = C.window_attention(qo[:, :, 3:67], s.cache, table, lengths, starts=starts, window=50, sinks=2, route="auto")
        direct = C.window_attention(q, s.cache, table, lengths, starts=starts, window=50, sinks=2, route="direct")
        assert torch.equal(got, direct)


def test_window_one_token_is_decode_attention():
    s = Streams(5, 700, 2, 128, 16, "bf16", True, seed=12)
    q = rand(5, 8, 128, scale=2).bfloat16().to(DEV)
    lengths = torch.tensor([700, 1, 0, 333, 64], dtype=torch.int32, device=DEV)
    a, la = C.window_attention(q, s.cache, s.table.to(DEV), lengths, lse=True)
    b, lb = C.decode_attention(q, s.cache, s.table.to(DEV), lengths, lse=True)
    # both within their bounds of the formula: half a step of the result each, and the weights' steps
    assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2.0 ** -10).all()
    assert torch.allclose(la, lb, atol=1e-4, rtol=0)


# ---------------------------------------------------------------- tree_attention


def random_tree(batch, drafts, seed):
    g = torch.Generator().manual_seed(seed)
    return ((torch.rand(batch, drafts, generator=g) * (torch.arange(drafts) + 1)).long() - 1)


def check_tree(streams, lengths, drafts, heads, tree, route="auto", scale=None, max_length=None, seed=0):
    s, dt = streams, streams.dt
    t = TYPES[dt]
    q = rand(s.batch, drafts, heads, s.dim, seed=seed + 13, scale=2).to(t)
    plan = C.tree_plan(s.cache, q.to(DEV), s.table.to(DEV), tree.to(DEV), scale, max_length, None, route)[1]
    print(f"tree {dt} q8 {s.cache.quantised} dim {s.dim} heads {heads} lengths {lengths} drafts {drafts} route {plan.route} chunks {plan.chunks}", flush=True)
    got, got_lse = C.tree_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), tree.to(DEV), scale=scale,
                                    max_length=max_length, lse=True, route=route)
    torch.cuda.synchronize()
    k, v, valid = s.tokens64("k"), s.tokens64("v"), s.page_seen()
    step = p_step(dt, s.cache.quantised, "direct" if plan.route == 1 else "mfma")
    real = s.dim ** -0.5 if scale is None else scale
    room = s.room if max_length is None else max_length
    for b in range(s.batch):
        words = (tree[b] if tree.dim() == 3 else tree).tolist()
        seen = torch.zeros(drafts, s.room, dtype=torch.bool)
        seen[:, :room] = tree_seen(min(lengths[b], room), drafts, room, words)
        seen &= valid[b]
        want, want_lse, mag, top = attend64(q[b], k[b], v[b], seen, real)
        most = int(seen.sum(1).max())
        within(got[b], want, row_bound(want, mag, top, s.dim, most, dt, step, s.cache.quantised), f"stream {b}")
        within(got_lse[b], want_lse, (2 * (s.dim + 12) * U * top + (most + 64) * U + 2.0 ** -17 + want_lse.abs().nan_to_num(0, 0, 0) * 4 * U), f"lse {b}")
    return got


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dt,quantised", [("bf16", False), ("bf16", True), ("f16", False), ("f16", True), ("f32", False), ("f32", True)])
@pytest.mark.parametrize("drafts,dim,page,heads,kv", [(1, 64, 16, 4, 2), (7, 128, 16, 8, 2), (25, 96, 32, 5, 1), (64, 64, 16, 2, 1), (65, 80, 16, 4, 2),
                                                      (130, 64, 48, 3, 3), (16, 256, 16, 4, 1), (9, 33, 7, 3, 1)])
def test_tree_types_and_sizes(route, dt, quantised, drafts, dim, page, heads, kv):
    s = Streams(3, 300, kv, dim, page, dt, quantised, seed=drafts)
    tree = C.tree_mask(random_tree(3, drafts, drafts))
    check_tree(s, [300 - drafts, 0, 77], drafts, heads, tree, route)


@pytest.mark.parametrize("route", ROUTES)
def test_tree_rows_that_see_nothing_stray_bits_and_shared_trees(route):
    s = Streams(3, 200, 1, 64, 16, "bf16", False, seed=20)
    drafts = 70
    g = torch.Generator().manual_seed(1)
    # any bits, in the words' unused ones too; some rows none
    tree = torch.randint(-2 ** 63, 2 ** 63 - 1, (3, drafts, 2), generator=g)
    tree[:, ::3] = 0
    check_tree(s, [0, 130, 64], drafts, 4, tree, route)
    check_tree(s, [-5, 0, 1], drafts, 4, tree[0], route)
    check_tree(s, [0, 0, 0], drafts, 4, torch.zeros_like(tree), route)
    # a tree whose rows and streams have strides of their own
    wide = torch.zeros(3, drafts, 5, dtype=torch.int64)
    wide[:, :, 1:3] = tree
    check_tree(s, [0, 130, 64], drafts, 4, wide[:, :, 1:3], route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("quantised", [False, True])
def test_tree_limits_pages_and_parts(route, quantised):
    s = Streams(2, 5000, 1, 64, 16, "f16", quantised, seed=21)
    tree = C.tree_mask(random_tree(2, 13, 5))
    check_tree(s, [4987, 2500], 13, 2, tree, route)
    # drafts past the table or max_length are left out
    check_tree(s, [4999, 5008], 13, 2, tree, route)
    check_tree(s, [10 ** 9, 2 ** 31 - 1], 13, 2, tree, route)
    check_tree(s, [95, 104], 13, 2, tree, route, max_length=100)
    check_tree(s, [95, 104], 13, 2, tree, route, max_length=0)
    s.table[0, 5], s.table[1, 156] = -1, 10 ** 6
    check_tree(s, [4987, 2500], 13, 2, tree, route)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dt,quantised", [("bf16", False), ("f16", False), ("bf16", True)])
def test_tree_bad_values_where_a_draft_does_not_see(route, dt, quantised):
    drafts = 40
    s = Streams(1, 128, 1, 64, 16, dt, quantised, seed=22)
    parents = random_tree(1, drafts, 9)
    tree = C.tree_mask(parents)
    for name in "kv":
        s.set(name, 0, 50 + 11, math.nan)
    for t in range(50 + drafts, s.room):
        s.set("v", 0, t, math.nan)
    q = rand(1, drafts, 2, 64, scale=2).to(TYPES[dt])
    got = C.tree_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor([50], dtype=torch.int32, device=DEV), tree.to(DEV), route=route).cpu()[0]
    sees = torch.tensor([bool(w[0] >> 11 & 1) for w in tree[0].tolist()])
    assert sees.any() and not sees.all()
    assert got[sees].isnan().all() and got[~sees].isfinite().all()


def test_tree_of_a_chain_is_a_window_without_limit():
    s = Streams(2, 400, 2, 64, 16, "bf16", False, seed=23)
    chain = C.tree_mask(torch.arange(-1, 19))
    q = rand(2, 20, 4, 64, scale=2).bfloat16().to(DEV)
    lengths = torch.tensor([380, 100], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 20, 40], dtype=torch.int32, device=DEV)
    for route in ROUTES:
        a = C.tree_attention(q, s.cache, s.table.to(DEV), lengths, chain.to(DEV), route=route)
        b = C.window_attention(q.view(40, 4, 64), s.cache, s.table.to(DEV), lengths + 20, starts=starts, route=route)
        assert ((a.view(40, 4, 64).float() - b.float()).abs() <= 2.0 ** -6 * b.float().abs() + 2.0 ** -9).all()


# ---------------------------------------------------------------- together


def test_prompt_then_drafts_together():
    """A prompt in two chunks, then a tree of drafts: append, window and tree over one cache, against
    64 bits from the same stored cells."""
    heads, kv, dim, page, batch = 4, 2, 64, 16, 2
    inv = freqs(dim // 2)
    for quantised in (False, True):
        s = Streams(batch, 160, kv, dim, page, "bf16", quantised, seed=30)
        table = s.table.to(DEV)
        done = [0, 0]
        for news in ([70, 33], [20, 50]):
            rows = sum(news)
            qkv = rand(rows, heads + 2 * kv, dim, seed=rows).bfloat16()
            pos = torch.cat([torch.arange(d, d + n) for d, n in zip(done, news)])
            who = torch.cat([torch.full((n,), b) for b, n in enumerate(news)])
            slots = C.cache_slots(table, who.to(DEV), pos.to(DEV), page)
            q, k, v = qkv.to(DEV).split([heads, kv, kv], 1)
            q = C.cache_append(s.cache, k, v, slots, pos.to(DEV), inv.to(DEV), q=q)
            done = [d + n for d, n in zip(done, news)]
            for name in "kv":
                s.host[name] = getattr(s.cache, name).cpu()
                if quantised:
                    s.scale[name] = getattr(s.cache, name + "_scale").cpu()
            check_window(s, done, news, heads, 40, 4, q=q.cpu())
        drafts = 9
        parents = random_tree(batch, drafts, 2)
        depth = torch.zeros(batch, drafts, dtype=torch.int64)
        for i in range(drafts):
            depth[:, i] = torch.where(parents[:, i] >= 0, depth.gather(1, parents[:, i:i + 1].clamp(min=0))[:, 0] + 1, 0)
        place = torch.tensor(done).view(-1, 1) + torch.arange(drafts)
        who = torch.arange(batch).view(-1, 1).expand(-1, drafts)
        slots = C.cache_slots(table, who.to(DEV), place.to(DEV), page).flatten()
        qkv = rand(batch * drafts, heads + 2 * kv, dim, seed=77).bfloat16().to(DEV)
        q, k, v = qkv.split([heads, kv, kv], 1)
        q = C.cache_append(s.cache, k, v, slots, (torch.tensor(done).view(-1, 1) + depth).flatten().to(DEV), inv.to(DEV), q=q)
        for name in "kv":
            s.host[name] = getattr(s.cache, name).cpu()
            if quantised:
                s.scale[name] = getattr(s.cache, name + "_scale").cpu()
        tree = C.tree_mask(parents)
        got = C.tree_attention(q.view(batch, drafts, heads, dim), s.cache, table, torch.tensor(done, dtype=torch.int32, device=DEV), tree.to(DEV))
        step = p_step("bf16", quantised, "mfma")
        k64, v64 = s.tokens64("k"), s.tokens64("v")
        for b in range(batch):
            seen = tree_seen(done[b], drafts, s.room, tree[b].tolist())
            want, _, mag, top = attend64(q.view(batch, drafts, heads, dim)[b].cpu(), k64[b], v64[b], seen, dim ** -0.5)
            within(got[b], want, row_bound(want, mag, top, dim, 200, "bf16", step, quantised), f"drafts of {b}")


@pytest.mark.parametrize("quantised", [False, True])
def test_calls_in_a_graph_and_on_another_stream(quantised):
    """A step of append, window and tree captured once and replayed on other inputs, with eager work between."""
    s = Streams(3, 3000, 1, 64, 16, "bf16", quantised, seed=31)
    table = s.table.to(DEV)
    heads, kv, dim = 2, 1, 64
    qkv = torch.zeros(3, heads + 2 * kv, dim, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(3, dtype=torch.int64, device=DEV)
    lengths = torch.zeros(3, dtype=torch.int32, device=DEV)
    tree = C.tree_mask(torch.tensor([-1, 0, 0])).to(DEV)
    inv = freqs(32).to(DEV)
    who = torch.arange(3, device=DEV)
    drafts = torch.zeros(3, 3, heads, dim, dtype=torch.bfloat16, device=DEV)

    def step():
        q, k, v = qkv.split([heads, kv, kv], 1)
        q = C.cache_append(s.cache, k, v, C.cache_slots(table, who, pos, 16), pos, inv, q=q)
        a = C.window_attention(q, s.cache, table, lengths, window=2500, sinks=4)
        b = C.tree_attention(drafts, s.cache, table, lengths, tree)
        return q, a, b

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for n in (5, 2900, 64, 1000):
        qkv.copy_(rand(3, 4, 64, seed=n))
        drafts.copy_(rand(3, 3, 2, 64, seed=n))
        pos.copy_(torch.tensor([n, n // 2, 0]))
        lengths.copy_(torch.tensor([n + 1, n // 2 + 1, 1]))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), n
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    q, k, v = qkv.split([heads, kv, kv], 1)
    a = C.cache_append(s.cache, k, v, C.cache_slots(table, who, pos, 16), pos, inv, q=q, stream=other)
    b = C.window_attention(want[0], s.cache, table, lengths, window=2500, sinks=4, stream=other.cuda_stream)
    c = C.tree_attention(drafts, s.cache, table, lengths, tree, stream=other)
    other.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, want[2])


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements (more than 2^32 bytes): the last pages are read and written where they are."""
    n = 2 ** 31 // (16 * 64) + 8
    cache = C.KVCache(torch.zeros(n, 1, 16, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(n, 1, 16, 64, dtype=torch.bfloat16, device=DEV))
    table = torch.tensor([[n - 1, 0, n - 3, 2]], dtype=torch.int32, device=DEV)
    k, v = rand(64, 1, 64).bfloat16().to(DEV), rand(64, 1, 64, seed=1).bfloat16().to(DEV)
    pos = torch.arange(64, device=DEV)
    slots = C.cache_slots(table, torch.zeros_like(pos), pos, 16)
    inv = freqs(32).to(DEV)
    small = C.KVCache.new(4, 1, 16, 64)
    q = rand(64, 2, 64, seed=2).bfloat16().to(DEV)
    a = C.cache_append(cache, k, v, slots, pos, inv, q=q)
    b = C.cache_append(small, k, v, pos, pos, inv, q=q)
    assert torch.equal(a, b)
    near = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4)
    length = torch.tensor([64], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 64], dtype=torch.int32, device=DEV)
    tree = C.tree_mask(torch.arange(-1, 7)).to(DEV)
    for route in ROUTES:
        x = C.window_attention(a, cache, table, length, starts=starts, window=20, sinks=2, route=route)
        y = C.window_attention(a, small, near, length, starts=starts, window=20, sinks=2, route=route)
        assert torch.equal(x, y)
        x = C.tree_attention(a[:8].view(1, 8, 2, 64), cache, table, length - 8, tree, route=route)
        y = C.tree_attention(a[:8].view(1, 8, 2, 64), small, near, length - 8, tree, route=route)
        assert torch.equal(x, y)
