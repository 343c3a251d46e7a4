"""GPU tests of the operators of several new tokens at the ends of their number ranges: values near the
largest of their type, positions far beyond 2^40."""
import math

import pytest
import torch

import convt_forward_amd as C
from tests.decode_util import U, rounding, within
from tests.extend_util import DEV, Streams, attend64, rand, rotated_bound, row_bound, tree_seen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("route", ["direct", "auto"])
@pytest.mark.parametrize("form", ["few rows", "128 rows", "256 rows"])
def test_values_near_the_largest(form, route):
    """A token whose score passes those before it by 2^7.2, less than what moves the base of the
    exponents, holds values near bfloat16's largest; all others hold zeros, and the result is finite."""
    batch, kv, drafts, share, room = {"few rows": (2, 1, 2, 4, 300), "128 rows": (2, 1, 25, 4, 300), "256 rows": (4, 8, 64, 4, 4700)}[form]
    s = Streams(batch, room, kv, 64, 16, "bf16", False, seed=90)
    for name in "kv":
        s.host[name].zero_()
    lengths = [room - drafts - 10 * b for b in range(batch)]
    at = 144  # in a later tile than the first one, of the same wave in the form for few rows too: its tiles of 32 tokens go round 4 waves
    for b in range(batch):
        page, off = int(s.table[b, at // 16]), at % 16
        s.host["k"][page, :, off, 0] = 5.0
        s.host["v"][page, :, off] = (torch.linspace(-1, 1, 64) * 3e38).bfloat16()
    for name in "kv":
        getattr(s.cache, name).copy_(s.host[name].to(DEV))
    q = torch.zeros(batch, drafts, kv * share, 64, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    tree = C.tree_mask(torch.arange(-1, drafts - 1))
    got, lse = C.tree_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), tree.to(DEV), scale=1.0,
                                lse=True, route=route)
    torch.cuda.synchronize()
    k, v = s.tokens64("k"), s.tokens64("v")
    for b in range(batch):
        seen = tree_seen(lengths[b], drafts, s.room, tree.tolist())[[0, drafts - 1]]
        want, want_lse, mag, top = attend64(q[b][[0, drafts - 1]], k[b], v[b], seen, 1.0)
        assert want.isfinite().all() and want.abs().max() > 1e36
        step = 0.0 if route == "direct" else 2.0 ** -8
        within(got[b][[0, drafts - 1]], want, row_bound(want, mag, top, 64, s.room, "bf16", step, False), f"stream {b}")


def append(positions, inv, q, interleaved=False):
    n = len(positions)
    cache = C.KVCache.new(-(-n // 16), 1, 16, q.shape[2], dtype=torch.float32)
    k = q[:, :1].contiguous().to(DEV)
    return C.cache_append(cache, k, k, torch.arange(n, device=DEV), positions.to(DEV), inv.to(DEV), q=q.to(DEV), interleaved=interleaved).cpu()


def test_append_positions_up_to_2_to_53():
    """Frequencies that are powers of two: the angle is exact in float64, and its sine and cosine are held
    to what they are near the first position."""
    half = 8
    inv = 2.0 ** -torch.arange(half, dtype=torch.float32)
    positions = torch.tensor([sign * (2 ** e - 3 * i) for e in (45, 48, 50, 51, 52, 53) for i in (0, 1, 7, 12345) for sign in (1, -1)])
    q = rand(len(positions), 2, 2 * half)
    turn = 10096689509235987743946820282484873672429286842977325943070736  # floor(2 pi 2^200)
    assert abs(turn / 2 ** 200 - 2 * math.pi) < 1e-15
    angle = torch.tensor([[((int(p) << (200 - i)) % turn) / 2 ** 200 for i in range(half)] for p in positions], dtype=torch.float64)
    a, b = q.double()[..., :half], q.double()[..., half:]
    c, s = angle.cos().unsqueeze(1), angle.sin().unsqueeze(1)
    want = torch.cat([a * c - b * s, a * s + b * c], -1)
    within(append(positions, inv, q), want, rounding(torch.float32, want) + rotated_bound((a.abs() + b.abs()).repeat(1, 1, 2)), "q")


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_turns_pairs_by_any_angle(interleaved):
    """Positions and frequencies whose angle is off by many turns (2^-52 of itself): a pair keeps its length."""
    half = 6
    inv = torch.tensor([1.0, 1000.0, -3e7, 1e15, 3e38, 1e-30])
    positions = torch.tensor([2 ** 63 - 1, -2 ** 63, 2 ** 60 + 12345, -2 ** 57, 2 ** 53 + 1, 10 ** 15])
    q = rand(len(positions), 3, 2 * half, seed=1)
    got = append(positions, inv, q, interleaved).double()

    def lengths(x):
        pair = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
        return pair[0].square() + pair[1].square()

    want = lengths(q.double())
    # sine and cosine are off by 2^-23 each, so the squares' sum of them by 2 sqrt(2) 2^-23; a dim's two products, its sum and
    # its rounding by 2^-24 each of |a| + |b| <= sqrt(2) times the length, which counts twice in the square
    within(lengths(got), want, want * (2 * 2 ** 0.5 * 2.0 ** -23 + 2 * 2 * 2 ** 0.5 * 4 * U), "length squared")


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("new,share", [(1, 4), (7, 2), (20, 4), (200, 2)])
def test_the_longest_stream(new, share, quantised):
    """A window at the end of 2^31 - 4097 tokens, and first tokens, is that of a short stream with the same pages there."""
    longest = 2 ** 31 - 4097
    s = Streams(1, 1024, 1, 64, 16, "bf16", quantised, seed=91)
    width = longest // 16 + 1
    table = torch.zeros(1, width, dtype=torch.int32, device=DEV)
    near = s.table.to(DEV)
    short = 40 * 16 + longest % 16
    table[:, :2] = near[:, :2]
    table[:, -40:] = near[:, 1:41]
    q = rand(new, share, 64, seed=5, scale=2).bfloat16().to(DEV)
    starts = torch.tensor([0, new], dtype=torch.int32, device=DEV)
    for route in ("direct", "auto"):
        for window, sinks in ((100, 0), (300, 3), (17, 20)):
            a = C.window_attention(q, s.cache, table, torch.tensor([longest], dtype=torch.int32, device=DEV), starts=starts, window=window, sinks=sinks,
                                   max_length=longest, lse=True, route=route)
            b = C.window_attention(q, s.cache, near, torch.tensor([short], dtype=torch.int32, device=DEV), starts=starts, window=window, sinks=sinks,
                                   lse=True, route=route)
            # the window begins as far into a page in both, so the same tokens share tiles
            assert all(torch.equal(x, y) for x, y in zip(a, b)), (route, window, sinks)
