"""GPU tests that the decoding-step operators compute in the precision they state: bounds by route
and type, each from the operations on the way of a term, so that operands or sums in
fewer bits do not pass. test_bounds_tell_fewer_bits shows that on the CPU."""
import math

import numpy as np
import pytest
import torch

import convt_forward_amd as C
from tests.decode_util import E4M3, TYPES, U, attend64, attend_bound, rounding, within

DEV = "cuda"


def q4_problem(rows, n, k, group, dt, x8):
    """x, x_scale, w, scales, and in 64 bits x, the scales and the weights before them, each [.., k]."""
    t, g = TYPES[dt], torch.Generator().manual_seed(rows + n + k + group)
    w = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = (0.02 * (0.5 + torch.rand(n, k // group, generator=g))).to(t)
    x, xs = torch.randn(rows, k, generator=g), None
    if x8:
        xs = x.abs().amax(-1) / 448
        x = (x / xs.unsqueeze(-1)).to(E4M3)
    else:
        x = x.to(t)
    x64 = x.double() * (1 if xs is None else xs.double().unsqueeze(-1))
    w64 = torch.stack([w & 15, w >> 4], -1).reshape(n, k).double() - 8
    return x, xs, w, scales, x64, scales.double().repeat_interleave(group, 1), w64


def q4_bound(x64, s64, w64, t, k, route):
    """Direct: a product, 8 of them added, the scale, k / 512 of these a lane, 6 joined, the row's scale.
    Matrix cores: the same terms with 15 in place of |w - 8|, since sums run over w and 8 is taken off
    afterwards; 128 products and their offset, the scale, k / 128 groups and 8 waves joined."""
    if route == "direct":
        mag, steps = x64.abs() @ (w64.abs() * s64).t(), k / 512 + 20
    else:
        mag, steps = x64.abs() @ s64.t() * 15, k / 128 + 64
    want = x64 @ (w64 * s64).t()
    return want, rounding(t, want) * (1 + 2.0 ** -6) + mag * steps * U


CASES = [("f32", False, "direct"), ("f32", True, "direct"), ("bf16", False, "direct"), ("f16", True, "direct"),
         ("bf16", False, "mfma"), ("f16", False, "mfma"), ("bf16", True, "mfma"), ("f16", True, "mfma")]


@pytest.mark.gpu
@pytest.mark.parametrize("dt,x8,route", CASES)
@pytest.mark.parametrize("rows,n,k,group", [(3, 37, 768, 32), (1, 50, 4096, 128), (20, 33, 1024, 64), (2, 9, 32, 32)])
def test_q4_precision(dt, x8, route, rows, n, k, group):
    x, xs, w, scales, x64, s64, w64 = q4_problem(rows, n, k, group, dt, x8)
    got = C.q4_matvec(x.to(DEV), w.to(DEV), scales.to(DEV), x_scale=None if xs is None else xs.to(DEV), route=route)
    want, bound = q4_bound(x64, s64, w64, TYPES[dt], k, route)
    within(got, want, bound, f"{dt} x8 {x8} {route}")


@pytest.mark.gpu
@pytest.mark.parametrize("group", [8, 256])
def test_q4_precision_of_other_groups(group):
    x, xs, w, scales, x64, s64, w64 = q4_problem(3, 37, 768, group, "f32", False)
    want, bound = q4_bound(x64, s64, w64, torch.float32, 768, "direct")
    within(C.q4_matvec(x.to(DEV), w.to(DEV), scales.to(DEV)), want, bound, f"f32 group {group}")


def attend_problem(dt, n, D, heads=4, kv=2):
    """q, k, v whose roundings to fewer bits all point one way, where random ones would cancel: the first token
    has weight 1 and value 0, every other one the weight and the value (per dim a power of two, of
    either sign) of almost 1 + 2^-11, which float16 cuts; scores come from one dim, so they are near exact."""
    t, odd = TYPES[dt], 1 + 0.49 * 2.0 ** -10
    q, k, v = torch.zeros(1, heads, D), torch.zeros(1, kv, n, D), torch.full((1, kv, n, D), odd)
    q[..., 0], k[:, :, 1:, 0] = 1, (math.log(odd) - 3 * math.log(2)) * D ** 0.5
    v *= torch.tensor([(-1.0) ** d * 2.0 ** (d % 3) for d in range(D)])
    v[:, :, 0] = 0
    return q.to(t), k.to(t), v.to(t)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,quantised,route,p_step", [
    ("f32", False, "direct", 8 * U), ("f32", True, "direct", 8 * U), ("bf16", False, "direct", 8 * U), ("f16", True, "direct", 8 * U),
    ("f16", False, "mfma", 2.0 ** -11), ("f16", True, "mfma", 2.0 ** -16), ("bf16", False, "mfma", 2.0 ** -16),
    ("bf16", True, "mfma", 2.0 ** -16)])
@pytest.mark.parametrize("n,D", [(5, 64), (100, 128), (700, 64), (3000, 128)])
def test_attend_precision(dt, quantised, route, p_step, n, D):
    """p meets V in float32 (direct: the power of two and at most two scalings of it, 8 u), in float16, or as
    the sum of two bfloat16 values; float16's smallest step is 2^-39 of the largest weight."""
    q, k, v = attend_problem(dt, n, D)
    t, width = TYPES[dt], -(-n // 16)
    cache = C.KVCache.new(width, 2, 16, D, dtype=t, quantised=quantised)
    table, at = torch.arange(width, dtype=torch.int32, device=DEV).view(1, width), torch.arange(n, device=DEV)
    C.cache_write(cache, k[0].transpose(0, 1).contiguous().to(DEV), v[0].transpose(0, 1).contiguous().to(DEV), at)
    # in float32, what a quantised cache holds: a code times its scale, one rounding
    k32, v32 = (x.cpu().transpose(0, 1).unsqueeze(0).double() for x in C.cache_read(cache, at, dtype=torch.float32 if quantised else t))
    out = C.decode_attention(q.to(DEV), cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale=D ** -0.5, route=route)
    want, _, mag, top = attend64(q, k32, v32, [n], D ** -0.5)
    bound = attend_bound(want, mag, top, D, n, t, p_step + 2 * U)
    if dt == "f16" and not quantised and route == "mfma":
        bound = bound + n * 2.0 ** -40 * v32.abs().max()
    within(out, want, bound, f"{dt} quantised {quantised} {route} {n} x {D}")


def test_bounds_tell_fewer_bits():
    """On the CPU: float32 arithmetic stays far inside the bounds of the direct kernels; a float32 problem with an
    operand or the weights rounded to float16 on the way leaves them."""
    for rows, n, k, group in [(3, 37, 768, 32), (3, 37, 768, 8), (1, 50, 4096, 128)]:
        x, _, _, scales, x64, s64, w64 = q4_problem(rows, n, k, group, "f32", False)
        want, bound = q4_bound(x64, s64, w64, torch.float32, k, "direct")

        def worst(x, s):
            return ((x.float() @ (w64.float() * s.float().repeat_interleave(group, 1)).t() - want).abs() / bound).max().item()
        assert worst(x, scales) < 0.3, (k, group)
        assert worst(x.half(), scales) > 2 and worst(x, scales.half()) > 2, (k, group)
    for n, D in [(100, 128), (700, 64)]:
        q, k, v = attend_problem("f32", n, D)
        want, _, mag, top = attend64(q, k.double(), v.double(), [n], D ** -0.5)
        bound = attend_bound(want, mag, top, D, n, torch.float32, 10 * U)

        def worst(p_type, o_type):
            s = torch.einsum("bhd,bhtd->bht", q, k.repeat_interleave(2, 1)) * D ** -0.5
            p = torch.exp(s - s.amax(-1, keepdim=True))
            out = torch.einsum("bht,bhtd->bhd", p.to(p_type).float(), v.repeat_interleave(2, 1).to(o_type).float()) / p.sum(-1, keepdim=True)
            return ((out - want).abs() / bound).max().item()
        assert worst(torch.float32, torch.float32) < 0.5, (n, D)
        assert worst(torch.float16, torch.float32) > 2 and worst(torch.float32, torch.float16) > 2, (n, D)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", sorted(TYPES))
def test_codes_and_scales_are_the_formula(dt):
    """s = max(max|r| / 448, 2^-126) and r * (1 / s) in float32, every division rounded to nearest, then the nearest
    code: bit for bit, at magnitudes from the scale's lower limit to the type's largest."""
    t = TYPES[dt]
    x = (rand := torch.randn(4000, 3, 80, generator=torch.Generator().manual_seed(5))).to(t)
    x[1::4] = (rand[1::4] * torch.finfo(t).smallest_normal * 64).to(t)
    x[2::4] = (rand[2::4].clamp(-4, 4) * (torch.finfo(t).max / 4)).to(t)
    x[3] = 0
    cache = C.KVCache.new(250, 3, 16, 80, quantised=True)
    C.cache_write(cache, x.to(DEV), x.to(DEV), torch.arange(4000, device=DEV))
    r = x.float().numpy()
    s = np.maximum(np.abs(r).max(-1) / np.float32(448), np.float32(2.0 ** -126))
    codes = torch.from_numpy(r * (np.float32(1) / s)[..., None]).to(E4M3)
    for held, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert np.array_equal(scale.cpu().transpose(1, 2).reshape(4000, 3).numpy(), s)
        assert torch.equal(held.cpu().view(torch.uint8).transpose(1, 2).reshape(4000, 3, 80), codes.view(torch.uint8))
