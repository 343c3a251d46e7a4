"""GPU tests of the decoding-step operators at the edges of what they accept: the longest lengths,
weights far below the largest, infinite values, rows that repeat in memory. Plain forms and
bounds are those of tests/decode_util.py."""
import math

import pytest
import torch

import convt_forward_amd as C
from tests.decode_util import TYPES, U, attend64, attend_bound, rounding, within

pytestmark = pytest.mark.gpu

DEV = "cuda"


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed + sum(shape)))


def one_stream(k, v, page=16):
    """A cache of one stream in scattered pages, its table and length; k and v [kv heads, tokens, dims]."""
    heads, n, dim = k.shape
    width = -(-n // page)
    cache = C.KVCache.new(width + 2, heads, page, dim, dtype=k.dtype)
    table = torch.randperm(width + 2, generator=torch.Generator().manual_seed(n))[:width].to(torch.int32).view(1, width).to(DEV)
    at = torch.arange(n, device=DEV)
    C.cache_write(cache, k.transpose(0, 1).contiguous().to(DEV), v.transpose(0, 1).contiguous().to(DEV),
                  C.cache_slots(table, torch.zeros_like(at), at, page))
    return cache, table, torch.tensor([n], dtype=torch.int32, device=DEV)


def test_attend_at_the_longest_length():
    """2^31 - 4097 tokens, the most a call takes, from one page that the table repeats. Every weight is the
    same, and 2^16 tokens of a page have the value 1, the others 0: all parts have to be joined."""
    page, ones, length = 2 ** 20, 2 ** 16, 2 ** 31 - 4097
    k = torch.zeros(1, 1, page, 16, device=DEV).bfloat16()
    v = torch.zeros_like(k)
    v[:, :, :ones] = 1
    table = torch.zeros(1, 2048, dtype=torch.int32, device=DEV)
    out, lse = C.decode_attention(torch.ones(1, 1, 16, device=DEV).bfloat16(), C.KVCache(k, v), table,
                                  torch.tensor([length], dtype=torch.int32, device=DEV), max_length=length, lse=True)
    # 2048 * 2^16 tokens of value 1; sums of whole numbers, 32768 parts joined, one rounding to bfloat16
    want = 2048 * ones / length
    assert ((out.double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -12)).all(), out
    assert abs(lse.item() - math.log(length)) <= 32 * 2.0 ** -20


@pytest.mark.parametrize("others", [1, 15, 100, 700])
@pytest.mark.parametrize("bits", [10, 14, 17, 20, 23, 24.7, 25.3, 28])
def test_attend_weights_far_below_the_largest(bits, others):
    """One token (of value 0) takes nearly all the weight; the others, each 2^-bits of it, carry the result."""
    D, t = 64, torch.float16
    q = torch.ones(1, 1, D, dtype=t)
    k, v = torch.zeros(1, 1, others + 1, D, dtype=t), 512 + 64 * rand(1, 1, others + 1, D).clamp(-3, 3)
    v = v.to(t)
    k[0, 0, 0], v[0, 0, 0] = bits * math.log(2) / D, 0
    cache, table, lens = one_stream(k[0], v[0])
    out = C.decode_attention(q.to(DEV), cache, table, lens, scale=1.0, route="mfma")
    want, _, mag, top = attend64(q, k.double(), v.double(), [others + 1], 1.0)
    # a weight is off by 2^-11 of itself, or by half of float16's smallest step where the largest is 2^15
    bound = attend_bound(want, mag, top, D, others + 1, t, 2.0 ** -11) + (others + 1) * 2.0 ** -40 * v.double().abs().max()
    within(out, want, bound, f"{others} weights of 2^-{bits}")


@pytest.mark.parametrize("route", ["auto", "direct"])
@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("n", [5, 100, 700])
def test_attend_infinite_values(dt, route, n):
    """An infinite value that is seen makes its dim of the result infinite, two of both signs make it NaN, a
    NaN NaN; all others stay as they are, and values past the length are not seen."""
    t, D = TYPES[dt], 64
    q, k, v = rand(1, 2, D, seed=1).to(t), (0.3 * rand(1, 1, n + 3, D, seed=2)).to(t), rand(1, 1, n + 3, D, seed=3).to(t)
    v[0, 0, 1, 3] = math.inf
    v[0, 0, n - 1, 17] = -math.inf
    v[0, 0, 0, 40], v[0, 0, n - 2, 40] = math.inf, -math.inf
    v[0, 0, n // 2, 50] = math.nan
    v[0, 0, 2, 60], v[0, 0, 3, 60] = torch.finfo(t).max / 8, -torch.finfo(t).max / 8
    v[0, 0, n:] = math.inf
    cache, table, _ = one_stream(k[0], v[0])
    out = C.decode_attention(q.to(DEV), cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale=D ** -0.5,
                             route=route).cpu()
    want, _, mag, top = attend64(q, k.double(), v.double(), [n], D ** -0.5)
    assert (want[0, :, 3] == math.inf).all() and (want[0, :, 17] == -math.inf).all() and want[0, :, [40, 50]].isnan().all()
    p_step = 2.0 ** -11 if dt == "f16" else 2.0 ** -15
    within(out, want, attend_bound(want, mag, top, D, n, t, p_step), f"{dt} {route} {n}")


def test_attend_refuses_a_workspace_it_would_write_past():
    cache, table, lens = one_stream(rand(2, 700, 64).bfloat16(), rand(2, 700, 64, seed=1).bfloat16())
    q = rand(1, 4, 64).bfloat16().to(DEV)
    need = C.attend_plan(cache, q, table)[1].workspace_bytes
    assert need > 0
    for bad in (torch.empty(1, dtype=torch.uint8, device=DEV).expand(need), torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2],
                torch.empty(need, dtype=torch.uint8), torch.empty(need - 1, dtype=torch.uint8, device=DEV)):
        with pytest.raises(ValueError, match="workspace"):
            C.decode_attention(q, cache, table, lens, workspace=bad)
    torch.cuda.synchronize()
    out = C.decode_attention(q, cache, table, lens, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    assert torch.equal(out, C.decode_attention(q, cache, table, lens))


@pytest.mark.parametrize("quantise", [False, True])
def test_norm_of_repeated_rows(quantise):
    """x and residual that are one row in memory for all rows (stride 0)."""
    x, r = rand(1, 200).bfloat16().to(DEV), rand(1, 200, seed=1).bfloat16().to(DEV)
    w = torch.ones(200, device=DEV).bfloat16()
    want = C.rms_norm(x.repeat(5, 1), w, residual=r.repeat(5, 1), quantise=quantise)
    got = C.rms_norm(x.expand(5, 200), w, residual=r.expand(5, 200), quantise=quantise)
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a.float(), b.float())


@pytest.mark.parametrize("route", ["auto", "direct"])
def test_q4_of_repeated_rows(route):
    w, s = (t.to(DEV) for t in C.q4_quantise(rand(50, 256).bfloat16(), 64))
    x = rand(1, 256, seed=2).bfloat16().to(DEV)
    for rows in (2, 20, 70):
        assert torch.equal(C.q4_matvec(x.expand(rows, 256), w, s, route=route), C.q4_matvec(x.repeat(rows, 1), w, s, route=route))


@pytest.mark.parametrize("route", ["auto", "direct"])
def test_attend_over_one_table_for_all_streams(route):
    n, D = 700, 64
    cache, table, _ = one_stream(rand(2, n, D).bfloat16(), rand(2, n, D, seed=1).bfloat16())
    q = rand(3, 4, D).bfloat16().to(DEV)
    lens = torch.tensor([n, 0, 33], dtype=torch.int32, device=DEV)
    got = C.decode_attention(q, cache, table.expand(3, table.shape[1]), lens, route=route)
    assert torch.equal(got, C.decode_attention(q, cache, table.repeat(3, 1), lens, route=route))


def test_tokens_without_a_place_are_not_written():
    cache = C.KVCache.new(4, 2, 16, 64)
    table = torch.tensor([[2, 1], [0, 3]], dtype=torch.int32, device=DEV)
    streams, positions = torch.tensor([0, 1, 0, 1], device=DEV), torch.tensor([-1, 32, 5, 10 ** 6], device=DEV)
    slots = C.cache_slots(table, streams, positions, 16)
    assert slots.tolist() == [-1, -1, 37, -1]
    k = rand(4, 2, 64).bfloat16().to(DEV)
    C.cache_write(cache, k, k, slots)
    assert torch.equal(cache.k[2, :, 5], k[2]) and torch.equal(cache.v[2, :, 5], k[2])
    cache.k[2, :, 5], cache.v[2, :, 5] = 0, 0
    assert (cache.k == 0).all() and (cache.v == 0).all()
    assert (C.cache_read(cache, slots)[0] == 0).all()


@pytest.mark.parametrize("rows,n", [(r, n) for r, most in ((7, 256), (16, 256), (17, 256), (32, 256), (33, 128), (64, 128), (65, 85), (130, 51))
                                    for n in (16 * most, 16 * most + 1, 32 * most + 3, 64 * most, 64 * most + 5)])
def test_q4_where_the_tiles_change(rows, n):
    """Both sides of the numbers of columns at which a wave takes 1, 2 or 4 tiles, and 8 or 4 waves share k."""
    k, group, t = 12288 if rows == 7 else 3200, 64, torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(rows + n)
    w = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = (0.02 * (0.5 + torch.rand(n, k // group, generator=g, device=DEV))).to(t)
    x = torch.randn(rows, k, generator=g, device=DEV).to(t)
    got = C.q4_matvec(x, w, s, route="auto")
    w64 = torch.stack([w & 15, w >> 4], -1).view(n, k).double() - 8
    s64 = s.double().repeat_interleave(group, 1)
    want = x.double() @ (w64 * s64).t()
    # sums run over w and 8 x: terms of at most 15 |x|
    bound = rounding(t, want) * (1 + 2.0 ** -6) + (x.double().abs() @ s64.t()) * (15 * (k / 128 + 64) * U)
    within(got, want.cpu(), bound.cpu(), f"{rows} x {k} x {n}")


@pytest.mark.parametrize("bits", [30.4, 33.6, 36.2, 38.7])
def test_attend_weights_below_the_relative_steps(bits):
    """Below 2^-29 of the largest a weight over a float16 cache is off by at most 2^-40, and not dropped."""
    D, t, others = 64, torch.float16, 500
    q = torch.ones(1, 1, D, dtype=t)
    k, v = torch.zeros(1, 1, others + 1, D, dtype=t), (50000 + 4000 * rand(1, 1, others + 1, D).clamp(-3, 3)).to(t)
    k[0, 0, 0], v[0, 0, 0] = bits * math.log(2) / D, 0
    cache, table, lens = one_stream(k[0], v[0])
    out = C.decode_attention(q.to(DEV), cache, table, lens, scale=1.0, route="mfma")
    want, _, mag, top = attend64(q, k.double(), v.double(), [others + 1], 1.0)
    bound = attend_bound(want, mag, top, D, others + 1, t, 2.0 ** -11) + others * 2.0 ** -40 * v.double().abs().max()
    assert (bound < want).all()  # 0 in its place would not pass
    within(out, want, bound, f"weights of 2^-{bits}")
