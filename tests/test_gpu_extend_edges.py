"""GPU tests of the edges of window_attention and tree_attention: every form of the matrix-core
kernel (few rows; 128 and 256 rows a block) with parts, rows that do not fill a block, infinite
values and missing pages in each, workspaces, unaligned pointers, calls at the same time, and that
the forms keep the precision they state."""
import math

import pytest
import torch

import convt_forward_amd as C
from tests.decode_util import TYPES, U, within
from tests.extend_util import DEV, Streams, attend64, rand, row_bound, tree_seen, window_seen
from tests.test_gpu_extend import check_tree, random_tree

pytestmark = pytest.mark.gpu


# rows of a stream (drafts x shared heads): up to 32, 128, more; and lengths that are cut into parts
@pytest.mark.parametrize("dt,quantised", [("bf16", False), ("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("drafts,share", [(4, 8), (8, 4), (33, 1), (25, 4), (128, 1), (33, 4), (40, 5), (64, 4), (65, 8)])
def test_forms_with_parts(dt, quantised, dim, drafts, share):
    s = Streams(2, 2600, 1, dim, 16, dt, quantised, seed=drafts + share)
    tree = C.tree_mask(random_tree(2, drafts, 3))
    assert C.tree_plan(s.cache, torch.zeros(2, drafts, share, dim, dtype=TYPES[dt], device=DEV), s.table.to(DEV), tree.to(DEV))[1].chunks > 1
    # the tree's rows are many and slow to check on the host: a few of them, of both ends
    q = rand(2, drafts, share, dim, seed=9, scale=2).to(TYPES[dt])
    lengths = [2600 - drafts, 700]
    got, lse = C.tree_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), tree.to(DEV), lse=True)
    torch.cuda.synchronize()
    k, v = s.tokens64("k"), s.tokens64("v")
    step = 2.0 ** -11 if quantised or dt == "f16" else 2.0 ** -8
    pick = sorted({0, 1, drafts // 2, drafts - 1})
    for b in range(2):
        seen = tree_seen(lengths[b], drafts, s.room, tree[b].tolist())[pick]
        want, want_lse, mag, top = attend64(q[b][pick], k[b], v[b], seen, dim ** -0.5)
        within(got[b][pick], want, row_bound(want, mag, top, dim, 2600, dt, step, quantised), f"stream {b}")
        within(lse[b][pick], want_lse, 2 * (dim + 12) * U * top + (2600 + 64) * U + 2.0 ** -17 + want_lse.abs() * 4 * U, f"lse {b}")


@pytest.mark.parametrize("new,share", [(1, 4), (7, 4), (20, 4), (60, 4), (150, 2), (300, 8)])
@pytest.mark.parametrize("quantised", [False, True])
def test_window_forms_ragged_with_parts(new, share, quantised):
    """One long stream among short and empty ones: parts by the real lengths, all rows checked against the direct kernel."""
    s = Streams(4, 5000, 1, 64, 16, "bf16", quantised, seed=new)
    lengths, news = [4990, 0, max(new // 2, 40), 900], [new, 0, new // 2, new]
    rows = sum(news)
    q = rand(rows + 3, share, 64, seed=1, scale=2).bfloat16().to(DEV)
    starts = torch.tensor([0] + news).cumsum(0).to(torch.int32).to(DEV)
    for window, sinks in ((None, 0), (3000, 70), (100, 2)):
        out = torch.full_like(q, 3.0)
        a, la = C.window_attention(q, s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), starts=starts, window=window,
                                   sinks=sinks, out=out, lse=True)
        b, lb = C.window_attention(q, s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), starts=starts, window=window,
                                   sinks=sinks, lse=True, route="direct")
        # the weights' steps (2^-8 of sum p |V|, and no |V| is above 5) and two roundings of the result
        assert ((a[:rows].float() - b[:rows].float()).abs() <= 2.0 ** -8 * 5 + 2.0 ** -7 * b[:rows].float().abs()).all(), (window, sinks)
        assert torch.allclose(la[:rows], lb[:rows], atol=2e-4, rtol=0)
        assert (out[rows:] == 3).all()


@pytest.mark.parametrize("share,dt,quantised", [(4, "bf16", False), (4, "bf16", True), (8, "f16", False), (1, "f16", True)])
def test_a_long_prompt_in_blocks_of_256_rows(share, dt, quantised):
    """Rows enough to fill the card with blocks of 256: missing pages, an infinite value that some rows see, a window and sinks."""
    new = 512 * 256 // (8 * share) + 37
    s = Streams(1, new + 50, 8, 64, 16, dt, quantised, seed=40)
    s.table[0, 3], s.table[0, s.table.shape[1] // 2] = -1, 10 ** 6
    far = new // 3
    s.set("v", 0, far, math.nan if quantised else math.inf)
    q = rand(new, 8 * share, 64, seed=2, scale=2).to(TYPES[dt])
    got = C.window_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor([new + 50], dtype=torch.int32, device=DEV),
                             starts=torch.tensor([0, new], dtype=torch.int32, device=DEV), window=300, sinks=20)
    torch.cuda.synchronize()
    k, v, valid = s.tokens64("k"), s.tokens64("v"), s.page_seen()
    first = far - 50  # the row at the position of the bad value
    pick = sorted({0, 1, first - 1, first, first + 150, first + 299, first + 300, new - 1, new // 2, 63, 64, 255, 256})
    p, t = torch.tensor(pick).view(-1, 1) + 50, torch.arange(s.room)
    seen = (t <= p) & ((t > p - 300) | (t < 20)) & valid[0]
    want, _, mag, top = attend64(q[pick], k[0], v[0], seen, 64 ** -0.5)
    step = 2.0 ** -11 if quantised or dt == "f16" else 2.0 ** -8
    within(got[pick], want, row_bound(want, mag, top, 64, 320, dt, step, quantised), "picked rows")
    bad = torch.zeros(new, dtype=torch.bool)
    bad[first:first + 300] = True
    assert got[~bad.to(DEV)].isfinite().all() and not got[bad.to(DEV)].isfinite().any()


@pytest.mark.parametrize("drafts,share", [(8, 2), (30, 4), (50, 4), (100, 4)])
@pytest.mark.parametrize("quantised", [False, True])
def test_forms_leave_out_pages_and_bad_values(drafts, share, quantised):
    s = Streams(2, 900, 1, 64, 16, "f16", quantised, seed=50 + drafts)
    s.table[0, 0], s.table[1, 7], s.table[0, 50] = -7, 10 ** 6, -1
    parents = random_tree(2, drafts, 4)
    tree = C.tree_mask(parents)
    s.set("v", 0, 700 + 3, math.nan)
    s.set("v", 1, 123 + 5, math.nan if quantised else -math.inf)
    for t in range(123 + drafts, 300):
        s.set("k", 1, t, math.nan)
    check_tree(s, [700, 123], drafts, share, tree)


@pytest.mark.parametrize("quantised", [False, True])
def test_few_rows_over_bfloat16_keep_more_than_8_bits_of_their_weights(quantised):
    """The form for few rows rounds a weight to the sum of two bfloat16 values (2^-16), or to float16 over
    e4m3 cells (2^-11). The values have random signs, so weights of one bfloat16 (2^-8) would make
    an error as large as the result's own rounding and independent of it: root 2 times that in the mean
    square; those of 2^-11 add 1 / 64 to the square. 10000 results tell these to a percent."""
    s = Streams(20, 64, 1, 64, 16, "bf16", quantised, seed=60)
    q = rand(20, 8, 64, seed=3, scale=2).bfloat16()
    lengths = torch.arange(20) + 45
    got = C.window_attention(q.to(DEV), s.cache, s.table.to(DEV), lengths.to(torch.int32).to(DEV)).cpu().double()
    k, v = s.tokens64("k"), s.tokens64("v")
    off, own = 0.0, 0.0
    for b in range(20):
        want = attend64(q[b:b + 1], k[b], v[b], window_seen(int(lengths[b]), 1, s.room, None, 0), 64 ** -0.5)[0]
        off += (got[b:b + 1] - want).square().sum().item()
        own += (want.bfloat16().double() - want).square().sum().item()
    print(f"error over that of one rounding: {(off / own) ** 0.5:.4f}", flush=True)
    assert off <= 1.15 ** 2 * own


@pytest.mark.parametrize("dt,quantised", [("bf16", False), ("f16", True)])
def test_256_rows_a_block_with_parts(dt, quantised):
    s = Streams(4, 4700, 8, 64, 16, dt, quantised, seed=61)
    drafts, lengths = 64, [4600, 3000, 0, 4636]
    s.table[1, 100] = -1
    s.set("v", 0, 4600 + 9, math.nan)
    tree = C.tree_mask(random_tree(4, drafts, 6))
    q = rand(4, drafts, 32, 64, seed=7, scale=2).to(TYPES[dt])
    got, lse = C.tree_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), tree.to(DEV), lse=True)
    assert C.tree_plan(s.cache, q.to(DEV), s.table.to(DEV), tree.to(DEV))[1].chunks > 1
    torch.cuda.synchronize()
    k, v, valid = s.tokens64("k"), s.tokens64("v"), s.page_seen()
    step = 2.0 ** -11 if quantised or dt == "f16" else 2.0 ** -8
    pick = [0, 9, 15, 16, 40, 63]
    for b in range(4):
        seen = (tree_seen(lengths[b], drafts, s.room, tree[b].tolist()) & valid[b])[pick]
        want, want_lse, mag, top = attend64(q[b][pick], k[b], v[b], seen, 64 ** -0.5)
        within(got[b][pick], want, row_bound(want, mag, top, 64, 4700, dt, step, quantised), f"stream {b}")
        within(lse[b][pick], want_lse, 2 * (64 + 12) * U * top + (4700 + 64) * U + 2.0 ** -17 + want_lse.abs() * 4 * U, f"lse {b}")
    sees = torch.tensor([bool(w[0] >> 9 & 1) for w in tree[0].tolist()])
    assert got[0].cpu()[sees].isnan().all() and got[0].cpu()[~sees].isfinite().all()


def test_workspaces():
    s = Streams(2, 5000, 1, 64, 16, "bf16", False, seed=70)
    table, lengths = s.table.to(DEV), torch.tensor([4900, 3000], dtype=torch.int32, device=DEV)
    q = rand(2, 9, 2, 64, scale=2).bfloat16().to(DEV)
    tree = C.tree_mask(torch.arange(-1, 8)).to(DEV)
    need = C.tree_plan(s.cache, q, table, tree)[1].workspace_bytes
    assert need > 0
    want = C.tree_attention(q, s.cache, table, lengths, tree)
    # what a workspace held before does not matter, nor that it is larger
    for fill in (0xff, 0x7f, 0x00):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(C.tree_attention(q, s.cache, table, lengths, tree, workspace=ws), want)
        assert (ws[need:] == fill).all()
    for bad in (torch.empty(need - 1, dtype=torch.uint8, device=DEV), torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2],
                torch.empty(1, dtype=torch.uint8, device=DEV).expand(need), torch.empty(need, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            C.tree_attention(q, s.cache, table, lengths, tree, workspace=bad)
    with pytest.raises(C.ConvtError):  # not 16-byte aligned
        C.tree_attention(q, s.cache, table, lengths, tree, workspace=torch.empty(need + 16, dtype=torch.uint8, device=DEV)[8:need + 8])


@pytest.mark.parametrize("quantised", [False, True])
def test_a_cache_that_is_not_aligned_runs_the_direct_kernel(quantised):
    t = torch.uint8 if quantised else torch.bfloat16
    s = Streams(2, 3000, 1, 64, 16, "bf16", quantised, seed=71)
    shape = s.cache.k.shape
    moved = {}
    for name in "kv":
        flat = torch.zeros(math.prod(shape) + 1, dtype=t, device=DEV)
        flat[1:] = getattr(s.cache, name).view(t).flatten()
        moved[name] = flat[1:].view(shape).view(getattr(s.cache, name).dtype)
    other = C.KVCache(moved["k"], moved["v"], s.cache.k_scale, s.cache.v_scale)
    q = rand(2, 9, 2, 64, scale=2).bfloat16().to(DEV)
    lengths = torch.tensor([2900, 1000], dtype=torch.int32, device=DEV)
    tree = C.tree_mask(torch.arange(-1, 8)).to(DEV)
    plan = C.tree_plan(other, q, s.table.to(DEV), tree)[1]
    assert plan.route == 2 and plan.chunks > 1
    a = C.tree_attention(q, other, s.table.to(DEV), lengths, tree)
    b = C.tree_attention(q, s.cache, s.table.to(DEV), lengths, tree, route="direct")
    # float32 both, in another order of parts; then the same rounding
    assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2.0 ** -14).all()


def test_two_calls_at_once():
    s = Streams(2, 4000, 1, 64, 16, "f16", False, seed=72)
    table, lengths = s.table.to(DEV), torch.tensor([3900, 2000], dtype=torch.int32, device=DEV)
    tree = C.tree_mask(torch.arange(-1, 8)).to(DEV)
    qs = [rand(2, 9, 2, 64, seed=i, scale=2).half().to(DEV) for i in range(4)]
    want = [C.tree_attention(q, s.cache, table, lengths, tree) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = []
        for q, st in zip(qs, streams):
            with torch.cuda.stream(st):
                got.append(C.tree_attention(q, s.cache, table, lengths, tree))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_closer_bound_gives_the_same():
    s = Streams(3, 3000, 1, 64, 16, "bf16", True, seed=73)
    q = rand(30, 4, 64, scale=2).bfloat16()
    starts = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([500, 77, 10], dtype=torch.int32, device=DEV)
    outs = [C.window_attention(q.to(DEV), s.cache, s.table.to(DEV), lengths, starts=starts, max_length=n) for n in (None, 1024, 512, 500)]
    for o in outs[1:]:
        assert ((o.float() - outs[0].float()).abs() <= 2.0 ** -7 * outs[0].float().abs() + 2.0 ** -11 * 4).all()


def test_decreasing_starts_stay_in_bounds():
    """starts that decrease or leave q give rows some result or none; rows of no stream and other memory stay."""
    s = Streams(4, 100, 1, 64, 16, "bf16", False, seed=74)
    lengths = torch.tensor([100, 90, 80, 70], dtype=torch.int32, device=DEV)
    for route in ("direct", "auto"):
        for share in (1, 40):
            base = torch.full((3 * 20, share, 64), 9.0, dtype=torch.bfloat16, device=DEV)
            q = rand(20, share, 64).bfloat16().to(DEV)
            for starts in ([0, 30, 10, 5, 20], [5, 4, 3, 2, 1], [-9, 2 ** 31 - 1, -5, 7, 20], [2 ** 31 - 1] * 5, [-2 ** 31, 0, 20, 20, 2 ** 31 - 1]):
                C.window_attention(q, s.cache, s.table.to(DEV), lengths, starts=torch.tensor(starts, dtype=torch.int64).to(torch.int32).to(DEV), window=9,
                                   out=base[20:40], route=route)
            torch.cuda.synchronize()
            assert (base[:20] == 9).all() and (base[40:] == 9).all()


def test_python_refusals():
    s = Streams(2, 100, 2, 64, 16, "bf16", False, seed=75)
    table, lengths = s.table.to(DEV), torch.tensor([90, 50], dtype=torch.int32, device=DEV)
    q = rand(2, 4, 64).bfloat16().to(DEV)

    def window(q=q, table=table, lengths=lengths, **kw):
        return C.window_attention(q, s.cache, table, lengths, **kw)

    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    window()
    window(starts=starts)
    for kw in [dict(window=0), dict(window=-3), dict(q=q[0]), dict(q=q[:, :, :32]), dict(q=q.cpu()), dict(table=table[0]), dict(table=table[:1]),
               dict(table=table.long()), dict(table=table.t().contiguous().t()), dict(lengths=lengths.long()), dict(lengths=lengths[:1]), dict(lengths=lengths.cpu()),
               dict(starts=starts[:2]), dict(starts=starts.long()), dict(starts=starts.cpu()), dict(out=q.float()), dict(out=q[:1]), dict(lse=torch.zeros(2, 3, device=DEV)),
               dict(lse=torch.zeros(2, 4)), dict(q=q.float()), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))]:
        with pytest.raises(ValueError):
            window(**kw)
    for kw in [dict(sinks=-1), dict(max_length=-1), dict(max_length=10 ** 6), dict(q=q[:, :3]), dict(scale=math.inf), dict(scale=math.nan)]:
        with pytest.raises(C.ConvtError):
            window(**kw)
    with pytest.raises(KeyError):
        window(route="fast")
    qt = rand(2, 5, 4, 64).bfloat16().to(DEV)
    tree = C.tree_mask(torch.arange(-1, 4)).to(DEV)

    def drafted(q=qt, tree=tree, **kw):
        return C.tree_attention(q, s.cache, table, lengths, tree, **kw)

    drafted()
    for kw in [dict(q=q), dict(tree=tree[:4]), dict(tree=tree.int()), dict(tree=tree.cpu()), dict(tree=tree.view(1, 5, 1)), dict(q=qt[:1]), dict(out=qt[:, :4])]:
        with pytest.raises(ValueError):
            drafted(**kw)
    k = rand(3, 2, 64).bfloat16().to(DEV)
    slots = torch.arange(3, device=DEV)
    inv = torch.ones(32, device=DEV)

    def append(k=k, v=k, slots=slots, positions=slots, inv=inv, q=None, **kw):
        return C.cache_append(s.cache, k, v, slots, positions, inv, q=q, **kw)

    q3 = rand(3, 4, 64).bfloat16().to(DEV)
    append(q=q3)
    for kw in [dict(positions=slots[:2]), dict(positions=slots.int()), dict(positions=slots.cpu()), dict(slots=slots.int()), dict(inv=inv.half()), dict(inv=torch.ones(33, device=DEV)),
               dict(inv=inv.view(1, 32)), dict(inv=inv.cpu()), dict(q=q3.half()), dict(q=q3[:2]), dict(q=q3[:, :0]), dict(q_out=q3), dict(q=q3, q_out=q3[:, :3]),
               dict(q=q3, q_out=q3.float()), dict(v=k[:2]), dict(k=k.float()), dict(inv=torch.ones(64, device=DEV)[::2])]:
        with pytest.raises(ValueError):
            append(**kw)
    # a refused call leaves no plan behind that a right one would find
    append(q=q3)


def test_nothing_to_do_and_nothing_to_see():
    q = rand(3, 4, 64).bfloat16().to(DEV)
    table, lengths = torch.zeros(3, 2, dtype=torch.int32, device=DEV), torch.full((3,), 20, dtype=torch.int32, device=DEV)
    tree = C.tree_mask(torch.arange(-1, 2)).to(DEV)
    # a cache without pages, and a page table without pages
    for cache, t in ((C.KVCache.new(0, 2, 16, 64), table), (C.KVCache.new(4, 2, 16, 64), table[:, :0])):
        for route in ("direct", "auto"):
            out, lse = C.window_attention(q, cache, t, lengths, lse=True, route=route)
            assert (out == 0).all() and (lse == -math.inf).all()
            out, lse = C.tree_attention(q.view(3, 1, 4, 64).expand(3, 3, 4, 64), cache, t, lengths, tree, lse=True, route=route)
            assert (out == 0).all() and (lse == -math.inf).all()
    cache = C.KVCache.new(4, 2, 16, 64)
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert C.window_attention(q[:0], cache, table[:0], lengths[:0]).shape == (0, 4, 64)
    assert C.window_attention(q[:0], cache, table[:0], lengths[:0], starts=none).shape == (0, 4, 64)
    assert C.window_attention(q[:0], cache, table, lengths, starts=torch.zeros(4, dtype=torch.int32, device=DEV)).shape == (0, 4, 64)
    assert C.tree_attention(q[:0].view(0, 1, 4, 64), cache, table[:0], lengths[:0], tree[:1]).shape == (0, 1, 4, 64)
    out = torch.full_like(q, 5.0)
    C.window_attention(q, cache, table[:0], lengths[:0], starts=none, out=out)  # rows of no stream
    torch.cuda.synchronize()
    assert (out == 5).all()


def test_repeated_rows_of_what_is_read():
    """A tree, a page table or queries given once for all streams, by strides of 0."""
    s = Streams(3, 300, 1, 64, 16, "bf16", False, seed=76)
    lengths = torch.tensor([200, 100, 280], dtype=torch.int32, device=DEV)
    tree = C.tree_mask(random_tree(1, 12, 1)).to(DEV)
    q = rand(1, 12, 4, 64, scale=2).bfloat16().to(DEV)
    table = s.table.to(DEV)[:1]
    for route in ("direct", "auto"):
        a = C.tree_attention(q.expand(3, -1, -1, -1), s.cache, table.expand(3, -1), lengths, tree.expand(3, -1, -1), route=route)
        b = C.tree_attention(q.repeat(3, 1, 1, 1), s.cache, table.repeat(3, 1), lengths, tree[0], route=route)
        assert torch.equal(a, b)
