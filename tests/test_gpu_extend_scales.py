"""GPU tests of window_attention and tree_attention over e4m3 caches whose value scales differ by many
binades: rows of zeros (scale 2^-126, or 0 where nothing was written yet), values far above others,
scales that are not numbers. Result and lse against 64 bits on both routes, in every form of the
matrix-core kernel, in one part and in several."""
import math

import pytest
import torch

import convt_forward_amd as C
from tests.decode_util import TYPES, U, within
from tests.extend_util import DEV, Streams, attend64, rand, row_bound, tree_seen, window_seen
from tests.test_gpu_extend import random_tree

pytestmark = pytest.mark.gpu


def edit(s, name, pages, offs, scale=None, factor=None, zero=False):
    """Codes and scales of the tokens (pages, offs), all heads, in the cache and in its copy."""
    if zero:
        s.host[name].view(torch.uint8)[pages, :, offs] = 0
    if scale is not None:
        s.scale[name][pages, :, offs] = scale
    if factor is not None:
        s.scale[name][pages, :, offs] *= factor.view(-1, 1)
    getattr(s.cache, name).copy_(s.host[name].to(DEV))
    getattr(s.cache, name + "_scale").copy_(s.scale[name].to(DEV))


def prepare(s, kind, lengths, dt):
    g = torch.Generator().manual_seed(5)
    for b, n in enumerate(lengths):
        t = torch.arange(s.room)
        if kind == "first tiles of zeros":
            t = t[:min(n, 256)]
        elif kind == "all but the last of zeros":
            t = t[:max(0, n - 2)]
        elif kind == "a part of zeros":
            t = t[n // 4:3 * n // 4]
        elif kind == "fresh places":
            t = t[torch.rand(s.room, generator=g) < 0.4]
        elif kind in ("first token", "a token of zeros", "a scale that is not a number", "an infinite scale"):
            t = t[:1]
        pages, offs = s.table[b, t // s.page].long(), t % s.page
        if kind in ("first tiles of zeros", "all but the last of zeros", "a part of zeros", "a token of zeros"):
            edit(s, "v", pages, offs, scale=2.0 ** -126, zero=True)
        elif kind == "first token":
            for name in "kv":
                edit(s, name, pages, offs, scale=2.0 ** -126, zero=True)
        elif kind == "fresh places":
            edit(s, "v", pages, offs, scale=0.0, zero=True)
        elif kind == "from 2^-126 to 1":
            edit(s, "v", pages, offs, scale=torch.exp2(torch.rand(len(t), 1, generator=g) * -126))
        elif kind == "from 2^-40 up":
            edit(s, "v", pages, offs, scale=torch.exp2(torch.rand(len(t), 1, generator=g) * (46 if dt == "f16" else 70) - 40))
        elif kind == "far above others":
            # values of 448 x 2^7 (float16) or 2^80, a zero row behind each of some of them
            f = torch.where(torch.rand(len(t), generator=g) < 0.1, 2.0 ** (12 if dt == "f16" else 87), 1.0)
            edit(s, "v", pages, offs, factor=f)
            edit(s, "v", pages[1::3], offs[1::3], scale=2.0 ** -126, zero=True)
        elif kind == "a scale that is not a number":
            edit(s, "v", pages, offs, scale=math.nan)
        elif kind == "an infinite scale":
            edit(s, "v", pages, offs, scale=math.inf, zero=True)


KINDS = ["first tiles of zeros", "all but the last of zeros", "a part of zeros", "fresh places", "first token", "a token of zeros", "from 2^-126 to 1", "from 2^-40 up",
         "far above others", "a scale that is not a number", "an infinite scale"]


def check_rows(s, got, got_lse, q, seen, step, what):
    """On the matrix cores a weight's exponent holds the logarithm of its value's scale, of up to 7
    bits before the point: its addition, the base's subtraction (half a step of 2^-17 each) and log2
    itself (a step of 2^-16) are off by 2^-15 in all, as is the softmax's sum, of as many roundings. A
    weight below 2^-60 of the row's largest may be left out."""
    k, v = s
    want, lse, mag, top = attend64(q, k, v, seen, q.shape[-1] ** -0.5)
    n = int(seen.sum(1).max())
    far = 2.0 ** -14 if step else 0.0
    largest = torch.stack([v[:, r].abs().nan_to_num(0, 0, 0).amax() if r.any() else torch.zeros((), dtype=torch.float64) for r in seen])
    bound = row_bound(want, mag, top, q.shape[-1], n, what[0], step, True) + mag * far + n * 2.0 ** -60 * largest.view(-1, 1, 1)
    within(got, want, bound, what[1])
    within(got_lse, lse, 2 * (q.shape[-1] + 12) * U * top + (n + 64) * U + 2.0 ** -17 + far + lse.abs().nan_to_num(0, 0, 0) * 4 * U, what[1] + " lse")


def run(kind, dt, route, s, lengths, news, heads, window, sinks, tree=None, chunks=None):
    prepare(s, kind, lengths, dt)
    print(f"{kind}, {dt}, lengths {lengths}, new {news}, heads {heads}, window {window}, sinks {sinks}, tree {tree is not None}", flush=True)
    table, at = s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV)
    rows = sum(news)
    q = rand(rows, heads, s.dim, seed=21, scale=2).to(TYPES[dt])
    if tree is None:
        starts = torch.tensor([0] + news).cumsum(0).to(torch.int32).to(DEV)
        plan = C.window_plan(s.cache, q.to(DEV), table, True, window, sinks, route=route)[1]
        got, lse = C.window_attention(q.to(DEV), s.cache, table, at, starts=starts, window=window, sinks=sinks, lse=True, route=route)
    else:
        qd = q.to(DEV).view(s.batch, news[0], heads, s.dim)
        plan = C.tree_plan(s.cache, qd, table, tree.to(DEV), route=route)[1]
        got, lse = C.tree_attention(qd, s.cache, table, at, tree.to(DEV), lse=True, route=route)
        got, lse = got.view(rows, heads, s.dim), lse.view(rows, heads)
    assert plan.route == (1 if route == "direct" else 2)
    if chunks is not None:
        assert (plan.chunks > 1) == chunks
    torch.cuda.synchronize()
    k, v = s.tokens64("k"), s.tokens64("v")
    done = 0
    for b, n in enumerate(news):
        pick = sorted({0, n // 3, n // 2, n - 1})
        seen = (window_seen(lengths[b], n, s.room, window, sinks) if tree is None else tree_seen(lengths[b], n, s.room, tree[b].tolist()))[pick]
        r = [done + i for i in pick]
        check_rows((k[b], v[b]), got[r], lse[r], q[r], seen, 0.0 if route == "direct" else 2.0 ** -11, (dt, f"stream {b}"))
        done += n


ROUTES = ["direct", "auto"]


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS)
def test_window_value_scales(kind, dt, route):
    for news, heads in (([1, 1], 4), ([7, 3], 4), ([20, 33], 4)):
        run(kind, dt, route, Streams(2, 700, 1, 64, 16, dt, True, seed=80), [690, 333], news, heads, 100, 1)
        run(kind, dt, route, Streams(2, 300, 1, 128, 16, dt, True, seed=81), [300, 290], news, heads, None, 0)
    # the only token
    run(kind, dt, route, Streams(2, 16, 1, 64, 16, dt, True, seed=82), [1, 1], [1, 1], 4, None, 0)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS)
def test_window_value_scales_over_parts(kind, dt, route):
    for news, heads in (([1, 1], 2), ([40, 30], 2)):
        run(kind, dt, route, Streams(2, 6000, 1, 64, 16, dt, True, seed=83), [5999, 4100], news, heads, None, 0, chunks=True if route == "auto" else None)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS)
def test_tree_value_scales(kind, dt, route):
    for drafts, share in ((7, 4), (25, 4)):
        tree = C.tree_mask(random_tree(2, drafts, 6))
        run(kind, dt, route, Streams(2, 300, 1, 96, 16, dt, True, seed=84), [250, 0], [drafts] * 2, share, None, 0, tree)
        run(kind, dt, route, Streams(2, 5000, 1, 64, 16, dt, True, seed=85), [4900, 2000], [drafts] * 2, share, None, 0, tree, chunks=True if route == "auto" else None)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS)
def test_value_scales_in_blocks_of_256_rows(kind, dt):
    tree = C.tree_mask(random_tree(4, 64, 6))
    run(kind, dt, "auto", Streams(4, 4700, 8, 64, 16, dt, True, seed=86), [4600, 3000, 0, 4636], [64] * 4, 32, None, 0, tree, chunks=True)
    new = 512 * 256 // (8 * 4) + 37
    run(kind, dt, "auto", Streams(1, new, 8, 64, 16, dt, True, seed=87), [new], [new], 32, 300, 1, chunks=False)


@pytest.mark.parametrize("drafts,share,batch,kv,room", [(7, 4, 2, 1, 300), (25, 4, 2, 1, 300), (25, 4, 2, 1, 3000), (64, 4, 4, 8, 4700)])
def test_what_lies_behind_a_stream_changes_no_bit(drafts, share, batch, kv, room):
    """Codes and scales behind the last token that a stream's rows see: unwritten places, NaN, infinities, garbage."""
    s = Streams(batch, room, kv, 64, 16, "bf16", True, seed=88)
    lengths = [room - drafts - 37 * (b + 1) for b in range(batch)]
    tree = C.tree_mask(random_tree(batch, drafts, 6))
    q = rand(batch, drafts, kv * share, 64, seed=22, scale=2).bfloat16().to(DEV)
    at = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    starts = torch.tensor([drafts * b for b in range(batch + 1)], dtype=torch.int32, device=DEV)
    first = None
    for scale, code in ((1.0, 0x38), (0.0, 0), (math.nan, 0x7f), (math.inf, 0xff), (-3.0, 0x01), (1e38, 0x7e), (1e-42, 0x80)):
        for b, n in enumerate(lengths):
            t = torch.arange(n + drafts, s.room)
            pages, offs = s.table[b, t // 16].long(), t % 16
            for name in "kv":
                s.host[name].view(torch.uint8)[pages, :, offs] = code
                s.scale[name][pages, :, offs] = scale
        for name in "kv":
            getattr(s.cache, name).copy_(s.host[name].to(DEV))
            getattr(s.cache, name + "_scale").copy_(s.scale[name].to(DEV))
        got = C.tree_attention(q, s.cache, s.table.to(DEV), at, tree.to(DEV), lse=True)
        got += C.window_attention(q.view(-1, kv * share, 64), s.cache, s.table.to(DEV), at + drafts, starts=starts, lse=True)
        first = got if first is None else first
        assert all(torch.equal(x, y) and x.isfinite().all() for x, y in zip(got, first)), scale
