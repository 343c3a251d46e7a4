"""The decoding-step operators, as cases to be measured: rms_norm, q4_matvec, cache_write /
cache_read and decode_attention. With `own` false `run` computes them from elementary torch
operations in float32; with `own` true it makes the calls that a user makes of the framework."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def listed():
    return [
        # one new token of one stream: the norm before a product that reads 8 bits
        dict(name="norm one token", op="norm", rows=1, width=1024, dtype="bf16", residual=True, quantise=True),
        # a ragged batch at an odd width, norm kept in 16 bits
        dict(name="norm odd batch", op="norm", rows=77, width=5001, dtype="f16", residual=True, quantise=False),
        # a long prompt
        dict(name="norm prompt", op="norm", rows=16384, width=8192, dtype="bf16", residual=True, quantise=True),
        # 64 streams, one new token each, into a quantised cache
        dict(name="write step", op="write", tokens=64, kv_heads=8, dim=128, page=16, pages=2048, dtype="bf16", quantised=True),
        # a prompt's keys and values, its length no multiple of the page
        dict(name="write prompt", op="write", tokens=32767, kv_heads=8, dim=128, page=64, pages=1024, dtype="f16", quantised=True),
        # a cached prefix read back in 16 bits
        dict(name="read prefix", op="read", tokens=65536, kv_heads=8, dim=128, page=64, pages=2048, dtype="bf16", quantised=True),
        # one stream's first tokens: latency
        dict(name="attend short", op="attend", batch=1, heads=8, kv_heads=2, dim=64, page=16, shortest=100, longest=100,
             dtype="bf16", quantised=False),
        # an ordinary batch of ragged streams with shared heads over an 8-bit cache
        dict(name="attend batch", op="attend", batch=32, heads=32, kv_heads=8, dim=128, page=16, shortest=1, longest=4096,
             dtype="bf16", quantised=True),
        # few streams over a long context: work has to be split over the length
        dict(name="attend long", op="attend", batch=4, heads=32, kv_heads=8, dim=128, page=64, shortest=100001, longest=131072,
             dtype="bf16", quantised=False),
        # one token through a square projection
        dict(name="matvec one token", op="matvec", rows=1, n=4096, k=4096, group=128, dtype="bf16", x8=False),
        # a small batch, odd output width, small groups
        dict(name="matvec odd batch", op="matvec", rows=7, n=10001, k=2560, group=32, dtype="f16", x8=False),
        # 16 streams through a wide projection, fed by the 8-bit norm
        dict(name="matvec wide", op="matvec", rows=16, n=32768, k=8192, group=128, dtype="bf16", x8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "write", "read", "attend", "attend", "matvec", "matvec"])
    if op == "norm":
        width = _log(rng, 16, 16384)
        return dict(op=op, rows=_log(rng, 1, min(16384, 2 ** 27 // width)), width=width, dtype=rng.choice(["bf16", "f16", "f32"]),
                    residual=rng.random() < 0.7, quantise=rng.random() < 0.5)
    if op in ("write", "read"):
        page = rng.choice([8, 16, 32, 64, 128])
        tokens, heads, dim = _log(rng, 1, 32768), rng.choice([1, 2, 4, 8]), rng.choice([32, 64, 80, 96, 128])
        return dict(op=op, tokens=tokens, kv_heads=heads, dim=dim, page=page, pages=-(-tokens // page) + rng.randrange(64),
                    dtype=rng.choice(["bf16", "f16", "f32"]), quantised=rng.random() < 0.7)
    if op == "attend":
        kv, share, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 96, 128, 256])
        batch = _log(rng, 1, 64)
        longest = _log(rng, 1, min(131072, 2 ** 28 // (batch * kv * dim)))
        return dict(op=op, batch=batch, heads=kv * share, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    shortest=rng.randrange(longest + 1), longest=longest, dtype=rng.choice(["bf16", "f16"]),
                    quantised=rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    n, k = _log(rng, 16, 32768), group * _log(rng, 1, 8192 // group)
    return dict(op=op, rows=_log(rng, 1, 32), n=n, k=k, group=group, dtype=rng.choice(["bf16", "f16"]), x8=rng.random() < 0.4)


def _lengths(c):
    """The streams' lengths, evenly from the longest to the shortest: the case alone fixes their sum."""
    b, lo, hi = c["batch"], c["shortest"], c["longest"]
    return [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]


def _quantise(x):
    """Rows of x (float32) in e4m3 and their scales."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
    return (x * (1.0 / scale).unsqueeze(-1)).to(E4M3), scale


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    s = dict(op=c["op"])
    if c["op"] == "norm":
        s["x"] = randn(c["rows"], c["width"]).to(t)
        s["residual"] = (3 * randn(c["rows"], c["width"])).to(t) if c["residual"] else None
        s["weight"] = (1 + 0.1 * randn(c["width"])).to(t)
        s["quantise"] = c["quantise"]
    elif c["op"] in ("write", "read"):
        shape = (c["pages"], c["kv_heads"], c["page"], c["dim"])
        for name in ("k", "v"):
            if c["quantised"]:
                s[name + "_cache"], s[name + "_scale"] = _quantise(randn(*shape))
            else:
                s[name + "_cache"], s[name + "_scale"] = randn(*shape).to(t), None
        slots = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:c["tokens"]]
        # pages are scattered, the tokens of a page follow each other
        pages = torch.randperm(c["pages"], generator=g, device=DEV)
        order = torch.arange(c["tokens"], device=DEV)
        s["slots"] = slots if c["tokens"] <= 256 else pages[order // c["page"]] * c["page"] + order % c["page"]
        s["dtype"] = t
        if c["op"] == "write":
            s["k"], s["v"] = (randn(c["tokens"], c["kv_heads"], c["dim"]).to(t) for _ in range(2))
    elif c["op"] == "attend":
        lengths = torch.tensor(_lengths(c), device=DEV, dtype=torch.int32)
        s["lengths"] = lengths[torch.randperm(c["batch"], generator=g, device=DEV)].contiguous()
        width = max(1, -(-c["longest"] // c["page"]))
        n_pages = c["batch"] * width
        s["page_table"] = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).view(c["batch"], width)
        s["q"] = (2 * randn(c["batch"], c["heads"], c["dim"])).to(t)
        s["scale"] = c["dim"] ** -0.5
        shape = (n_pages, c["kv_heads"], c["page"], c["dim"])
        for name in ("k", "v"):
            if c["quantised"]:
                s[name + "_cache"], s[name + "_scale"] = _quantise(randn(*shape))
            else:
                s[name + "_cache"], s[name + "_scale"] = randn(*shape).to(t), None
    else:
        x = randn(c["rows"], c["k"])
        s["x"], s["x_scale"] = _quantise(x) if c["x8"] else (x.to(t), None)
        s["w"] = torch.randint(0, 256, (c["n"], c["k"] // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["scales"] = (0.01 * (0.5 + torch.rand((c["n"], c["k"] // c["group"]), generator=g, device=DEV))).to(t)
    return s


def _cache(s):
    """The framework's handle of a cache, kept in the state as a program keeps it."""
    if "cache" not in s:
        import convt_forward_amd as C
        s["cache"] = C.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s["cache"]


def _own(s):
    import convt_forward_amd as C
    if s["op"] == "norm":
        return C.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6, quantise=s["quantise"])
    if s["op"] == "write":
        C.cache_write(_cache(s), s["k"], s["v"], s["slots"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if s["op"] == "read":
        return C.cache_read(_cache(s), s["slots"], dtype=s["dtype"])
    if s["op"] == "attend":
        return C.decode_attention(s["q"], _cache(s), s["page_table"], s["lengths"], scale=s["scale"])
    return C.q4_matvec(s["x"], s["w"], s["scales"], x_scale=s["x_scale"])


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    out = h.to(s["x"].dtype) if s["residual"] is not None else None
    if s["quantise"]:
        return (*_quantise(y), out)
    return y.to(s["x"].dtype), None, out


def _plain_write(s):
    page = s["k_cache"].shape[2]
    at, off = s["slots"] // page, s["slots"] % page
    for name in ("k", "v"):
        x = s[name]
        if s[name + "_scale"] is not None:
            x, scale = _quantise(x.float())
            s[name + "_scale"][at, :, off] = scale
            s[name + "_cache"].view(torch.uint8)[at, :, off] = x.view(torch.uint8)
        else:
            s[name + "_cache"][at, :, off] = x
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_read(s):
    page = s["k_cache"].shape[2]
    at, off = s["slots"] // page, s["slots"] % page

    def read(cache, scale):
        if scale is None:
            return cache[at, :, off].to(s["dtype"])
        x = cache.view(torch.uint8)[at, :, off].view(E4M3).float()
        return (x * scale[at, :, off].unsqueeze(-1)).to(s["dtype"])

    return read(s["k_cache"], s["k_scale"]), read(s["v_cache"], s["v_scale"])


def _plain_attend(s):
    q, table = s["q"], s["page_table"].long()
    batch, heads, dim = q.shape
    kv = s["k_cache"].shape[1]

    def gather(cache, scale):
        x = cache.view(torch.uint8)[table].view(E4M3).float() * scale[table].unsqueeze(-1) if scale is not None else cache[table].float()
        return x.transpose(1, 2).reshape(batch, kv, -1, dim)

    k = gather(s["k_cache"], s["k_scale"])
    score = torch.matmul(q.float().view(batch, kv, heads // kv, dim) * s["scale"], k.transpose(-1, -2))
    del k
    seen = torch.arange(score.shape[-1], device=q.device) < s["lengths"].view(batch, 1, 1, 1)
    top = score.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(top.isinf(), 0.0, top)), 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, gather(s["v_cache"], s["v_scale"])) / torch.where(total > 0, total, 1.0)
    return out.reshape(batch, heads, dim).to(q.dtype)


def _plain_matvec(s):
    n, groups = s["scales"].shape
    w = torch.stack([s["w"] & 15, s["w"] >> 4], -1).view(n, groups, -1).float() - 8
    w = (w * s["scales"].float().unsqueeze(-1)).view(n, -1)
    y = torch.matmul(s["x"].float(), w.t())
    if s["x_scale"] is not None:
        y = y * s["x_scale"].unsqueeze(-1)
    return y.to(s["scales"].dtype)


PLAIN = {"norm": _plain_norm, "write": _plain_write, "read": _plain_read, "attend": _plain_attend, "matvec": _plain_matvec}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}[c["dtype"]]
    if c["op"] == "norm":
        n = c["rows"] * c["width"]
        per = size + (2 * size if c["residual"] else 0) + (1 if c["quantise"] else size)
        return {"bytes": n * per + c["width"] * size + (4 * c["rows"] if c["quantise"] else 0), "flops": 6 * n}
    if c["op"] in ("write", "read"):
        rows = 2 * c["tokens"] * c["kv_heads"]
        cell = c["dim"] + 4 if c["quantised"] else c["dim"] * size
        return {"bytes": rows * (c["dim"] * size + cell) + 8 * c["tokens"], "flops": 3 * rows * c["dim"] if c["quantised"] else 0}
    if c["op"] == "attend":
        total = sum(_lengths(c))
        cell = c["dim"] + 4 if c["quantised"] else c["dim"] * size
        pages = sum(-(-n // c["page"]) for n in _lengths(c))
        return {"bytes": 2 * total * c["kv_heads"] * cell + 2 * c["batch"] * c["heads"] * c["dim"] * size + 4 * pages + 4 * c["batch"],
                "flops": 4 * total * c["heads"] * c["dim"]}
    x = c["rows"] * (c["k"] + 4 if c["x8"] else c["k"] * size)
    return {"bytes": c["n"] * c["k"] // 2 + size * c["n"] * (c["k"] // c["group"]) + x + size * c["rows"] * c["n"],
            "flops": 2 * c["rows"] * c["n"] * c["k"]}


# In 64 bits. Values held in e4m3 are given before their rounding: the error of both sides
# is then the format's own.


def _exact_cells(x):
    s = torch.clamp(x.abs().max(dim=-1).values / 448, min=2.0 ** -126)
    return x / s[..., None], s


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        d = x.shape[1]
        y = x / ((x * x).sum(1, keepdim=True) / d + 1e-6).sqrt() * s["weight"].double()[None]
        r = x if s["residual"] is not None else None
        return (*_exact_cells(y), r) if s["quantise"] else (y, None, r)
    if op in ("write", "read"):
        pages, heads, page, dim = s["k_cache"].shape
        found = []
        scales = []
        for name in ("k", "v"):
            flat = s[name + "_cache"].double().permute(0, 2, 1, 3).reshape(pages * page, heads, dim)
            sc = s[name + "_scale"]
            if sc is not None:
                sc = sc.double().permute(0, 2, 1).reshape(pages * page, heads)
            if op == "read":
                rows = flat.index_select(0, s["slots"])
                found.append(rows if sc is None else rows * sc.index_select(0, s["slots"])[..., None])
                continue
            new = s[name].double()
            if sc is not None:
                new, new_scale = _exact_cells(new)
                sc = sc.index_copy(0, s["slots"], new_scale).view(pages, page, heads).permute(0, 2, 1).contiguous()
            found.append(flat.index_copy(0, s["slots"], new).view(pages, page, heads, dim).permute(0, 2, 1, 3).contiguous())
            scales.append(sc)
        return tuple(found + scales)
    if op == "attend":
        q = s["q"].double()
        out = torch.zeros_like(q)
        share = case["heads"] // case["kv_heads"]
        for b, n in enumerate(s["lengths"].tolist()):
            if n == 0:
                continue
            ids = s["page_table"][b, :-(-n // case["page"])].long()
            for h in range(case["kv_heads"]):
                k, v = (s[m + "_cache"][:, h].view(torch.uint8 if case["quantised"] else s["k_cache"].dtype)[ids] for m in "kv")
                if case["quantised"]:
                    k, v = (a.view(E4M3).double() * s[m + "_scale"][:, h][ids].double()[..., None] for a, m in ((k, "k"), (v, "v")))
                k, v = (a.double().reshape(-1, case["dim"])[:n] for a in (k, v))
                p = torch.softmax((k @ q[b, h * share:(h + 1) * share].t()) * s["scale"], dim=0)
                out[b, h * share:(h + 1) * share] = p.t() @ v
        return out
    k = case["k"]
    w = torch.empty((case["n"], k), dtype=torch.float64, device=s["w"].device)
    w[:, 0::2] = (s["w"] % 16).double() - 8
    w[:, 1::2] = torch.div(s["w"], 16, rounding_mode="floor").double() - 8
    w *= s["scales"].double().repeat_interleave(case["group"], dim=1)
    x = s["x"].double() * (1 if s["x_scale"] is None else s["x_scale"].double()[:, None])
    return x @ w.t()
