"""Plain 64-bit forms of the decoding-step operators and the error bounds that the tests hold
the kernels to. The bounds are derived, not fitted:

  half(t)    a rounding to type t is off by at most half a step, torch.finfo(t).eps / 2 of
             the value, or half the smallest subnormal below the normal range;
  u = 2^-24  a float32 operation's relative rounding; a float32 sum of n terms in any order is
             off by at most n u times the sum of their magnitudes.
"""
import math

import torch

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rounding(t, value):
    """The bound on one rounding of `value` (float64) to type t."""
    f = torch.finfo(t)
    return torch.maximum(value.abs() * (f.eps / 2), torch.full_like(value, f.smallest_normal * f.eps / 2))


def within(got, want, bound, what=""):
    """got is within bound of want everywhere (NaN where want is NaN, equal where it is infinite)."""
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = ~want.isnan() & ~inf
    off = (got - want).abs()[fine]
    lim = bound.expand_as(want)[fine]
    if off.numel():
        worst = (off / lim.clamp(min=1e-300)).max().item()
        print(f"  {what}: worst {worst:.3f} of the bound", flush=True)
        assert (off <= lim).all(), f"{what}: {worst} times the bound"


def quantised_bound(r, s):
    """The bound on q * s against the row r (float64, [..., d]) with scale s ([...]): half an e4m3
    step (2^-4 of the value, 2^-10 of the scale below the normal range), and the
    float32 roundings of r / s (3 of them) on top."""
    s = s.unsqueeze(-1)
    return torch.maximum(r.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -10) + r.abs() * 4 * U


def norm64(x, weight, residual, eps):
    h = x.double() + (residual.double() if residual is not None else 0)
    y = h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    return y, h


def attend64(q, k, v, lengths, scale, seen=None):
    """q [B, H, D], k and v [B, HKV, L, D] (float64): out, lse, and A = sum p |V| and the largest
    sum |scale q k| of each (stream, head) for the bounds."""
    B, H, D = q.shape
    g = H // k.shape[1]
    out, mag = torch.zeros(B, H, D, dtype=torch.float64), torch.zeros(B, H, D, dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64)
    top = torch.zeros(B, H, dtype=torch.float64)
    for b in range(B):
        n = int(lengths[b])
        at = torch.arange(max(0, n))
        if seen is not None:
            at = at[seen[b, :max(0, n)]]
        if len(at) == 0:
            continue
        for h in range(H):
            kk, vv = k[b, h // g, at], v[b, h // g, at]
            s = kk @ q[b, h].double() * scale
            lse[b, h] = torch.logsumexp(s, 0)
            p = torch.softmax(s, 0)
            out[b, h] = p @ vv
            mag[b, h] = p @ vv.abs()
            top[b, h] = (kk.abs() @ q[b, h].double().abs()).max() * abs(scale)
    return out, lse, mag, top


def attend_bound(out, mag, top, D, n, t, p_step):
    """Errors of the scores shift every p by at most e^(2 ds) - 1 with ds = (D + 8) u
    times the largest sum of magnitudes (and 4 u |s| for the scaling and the power of
    two); p itself is held to p_step of its value where it meets V (and to its
    type's smallest step, 2^-25 a token at float16); sums over n tokens add n / 4 + 64
    roundings (4 waves share them); the result is rounded once."""
    ds = (D + 12) * U * top.unsqueeze(-1)
    rel = 2 * ds + p_step + (n / 4 + 64) * U
    return mag * rel * (1 + 2.0 ** -6) + rounding(t, out) * (1 + 2.0 ** -6)
