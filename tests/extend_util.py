"""Plain 64-bit forms of the operators of several new tokens per stream, on the host. The bounds
are those of tests/decode_util.py; what is added is derived here."""
import math

import torch

import convt_forward_amd as C
from tests.decode_util import E4M3, TYPES, U, rounding

DEV = "cuda"


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 1000 * len(shape) + sum(shape))
    return torch.randn(*shape, generator=g) * scale


def rotate64(x, positions, inv_freq, interleaved):
    """x [tokens, heads, dim] (float64) rotated, and for each element |a| + |b| of its pair (0 where it stays)."""
    half = inv_freq.shape[0]
    y, mag = x.clone(), torch.zeros_like(x)
    angle = positions.double().view(-1, 1, 1) * inv_freq.double()
    i = torch.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., one], x[..., two]
    y[..., one] = a * angle.cos() - b * angle.sin()
    y[..., two] = a * angle.sin() + b * angle.cos()
    mag[..., one] = mag[..., two] = a.abs() + b.abs()
    return y, mag


def rotated_bound(mag, angle_off=0.0):
    """Sine and cosine are off by at most 2^-23 (their polynomials' roundings and the argument's,
    2^-24 of at most pi / 4) plus what the angle itself is off by; two products and a sum in
    float32 add 2 roundings of each term."""
    return mag * (2.0 ** -23 + 2 * U + angle_off) * (1 + 2.0 ** -10)


class Streams:
    """A paged cache with the tokens of `batch` streams in scattered pages, on the device, and the
    same tokens in 64 bits on the host (k, v [batch, kv_heads, room, dim])."""

    def __init__(self, batch, room, kv_heads, dim, page, dt, quantised, seed=0, spare=2, layout="head", scale=1.0):
        t = TYPES[dt]
        self.batch, self.dim, self.page, self.dt = batch, dim, page, dt
        width = max(1, -(-room // page))
        self.room = width * page
        n = batch * width + spare
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(n, generator=g)[:batch * width].to(torch.int32).view(batch, width)
        self.host, self.scale = {}, {}
        device = {}
        for j, name in enumerate("kv"):
            x = rand(n, kv_heads, page, dim, seed=seed + 7 + j, scale=scale)
            if quantised:
                s = (x.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
                x = (x / s.unsqueeze(-1)).to(E4M3)
                self.scale[name] = s
                self.host[name] = x
            else:
                x = x.to(t)
                self.host[name] = x
                self.scale[name] = None
            if layout == "token":  # [page, token, head, dim] in memory
                device[name] = x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
            else:
                device[name] = x.to(DEV)
        dev = {k: None if s is None else s.to(DEV) for k, s in self.scale.items()}
        self.cache = C.KVCache(device["k"], device["v"], dev["k"], dev["v"])

    def set(self, name, b, t, value):
        """Put a value into every dim of token t of stream b, in cache and copy."""
        page, off = int(self.table[b, t // self.page]), t % self.page
        self.host[name][page, :, off] = torch.tensor(value).to(self.host[name].dtype)
        getattr(self.cache, name)[page, :, off] = torch.tensor(value).to(self.host[name].dtype).to(DEV)

    def tokens64(self, name):
        x = self.host[name].double()
        if self.scale[name] is not None:
            x = x * self.scale[name].double().unsqueeze(-1)
        valid = self.table.clamp(0, x.shape[0] - 1).long()
        return x[valid].transpose(1, 2).reshape(self.batch, x.shape[1], self.room, self.dim)

    def page_seen(self):
        n = self.host["k"].shape[0]
        return ((self.table >= 0) & (self.table < n)).repeat_interleave(self.page, 1)


def attend64(q, k, v, seen, scale):
    """q [n, H, D], k and v [HKV, L, D], seen [n, L]: out, lse, sum p |V|, the largest sum |scale q k|."""
    n, H, D = q.shape
    share = H // k.shape[0]
    out, mag = torch.zeros(n, H, D, dtype=torch.float64), torch.zeros(n, H, D, dtype=torch.float64)
    lse, top = torch.full((n, H), -math.inf, dtype=torch.float64), torch.zeros(n, H, dtype=torch.float64)
    for i in range(n):
        at = seen[i].nonzero().flatten()
        if len(at) == 0:
            continue
        kk, vv = k[:, at].repeat_interleave(share, 0), v[:, at].repeat_interleave(share, 0)
        s = torch.matmul(kk, q[i].double().unsqueeze(-1)).squeeze(-1) * scale
        lse[i] = torch.logsumexp(s, -1)
        p = torch.softmax(s, -1).unsqueeze(1)
        out[i] = torch.matmul(p, vv).squeeze(1)
        mag[i] = torch.matmul(p, vv.abs()).squeeze(1)
        top[i] = torch.matmul(kk.abs(), q[i].double().abs().unsqueeze(-1)).squeeze(-1).amax(-1) * abs(scale)
    return out, lse, mag, top


def p_step(dt, quantised, route):
    """How far a weight may be rounded where it meets V on the matrix cores: to float16 (2^-11)
    for float16 and e4m3 caches, to bfloat16 (2^-8) for bfloat16 ones; float32 on the direct route."""
    if route == "direct" or dt == "f32":
        return 0.0
    return 2.0 ** -11 if quantised or dt == "f16" else 2.0 ** -8


def row_bound(out, mag, top, D, n, dt, step, quantised):
    """attend_bound of decode_util with the weights' step. With e4m3 on the matrix cores a weight
    carries the logarithm of its value's scale, off by a rounding of its size (at most 2^-17 for one
    of up to 2^6 binades), and weights in float16 below 2^-14 / 2^7 of the largest are off by
    2^-32 of it each."""
    ds = (D + 12) * U * top.unsqueeze(-1) + (2.0 ** -17 if quantised and step else 0.0)
    rel = 2 * ds + step + (n / 4 + 64) * U
    tiny = n * 2.0 ** -32 * 2 if step == 2.0 ** -11 else 0.0
    return mag * (rel * (1 + 2.0 ** -6)) + tiny * mag.amax(-1, keepdim=True) + rounding(TYPES[dt], out) * (1 + 2.0 ** -6)


def window_seen(length, n, room, window, sinks):
    """[n, room]: what the last n of `length` tokens see."""
    p = torch.arange(length - n, length).view(-1, 1)
    t = torch.arange(room)
    seen = t <= p
    if window:
        seen &= (t > p - window) | (t < sinks)
    return seen


def tree_seen(length, drafts, room, rows):
    """[drafts, room] for the rows (lists of words) of one stream's tree."""
    seen = torch.zeros(drafts, room, dtype=torch.bool)
    seen[:, :max(0, min(length, room))] = True
    for i, words in enumerate(rows):
        for j in range(drafts):
            if words[j // 64] >> (j % 64) & 1 and max(0, length) + j < room:
                seen[i, max(0, length) + j] = True
    return seen
