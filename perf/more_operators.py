"""The operators of steps with several new tokens per stream, as cases to be measured:
cache_append, window_attention and tree_attention. With `own` false `run` computes them from
elementary torch operations in float32 (angles in float64); with `own` true it makes the calls
that a user makes of the framework."""
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
        # the next token of one stream: latency
        dict(name="append one token", op="append", tokens=1, heads=8, kv_heads=2, dim=64, rotary=64, interleaved=False, page=16, pages=64,
             first=100, dtype="bf16", quantised=False),
        # 64 streams, one new token each, into an 8-bit cache
        dict(name="append step", op="append", tokens=64, heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False, page=16, pages=2048,
             first=4000, dtype="bf16", quantised=True),
        # an odd chunk of a prompt, part of each head rotated in neighbouring pairs
        dict(name="append odd chunk", op="append", tokens=1531, heads=20, kv_heads=4, dim=96, rotary=64, interleaved=True, page=16, pages=128,
             first=77, dtype="f16", quantised=False),
        # the last chunk of a long document, far from the first position
        dict(name="append prompt", op="append", tokens=32767, heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False, page=64, pages=1024,
             first=98305, dtype="bf16", quantised=True),
        # a short window of one stream, one token: latency
        dict(name="window one token", op="window", batch=1, new=1, heads=8, kv_heads=2, dim=64, page=16, shortest=1000, longest=1000, window=256,
             sinks=4, dtype="bf16", quantised=False),
        # 64 streams of all lengths, one new token each, over an 8-bit cache
        dict(name="window step", op="window", batch=64, new=1, heads=32, kv_heads=8, dim=128, page=16, shortest=1, longest=32768, window=4096,
             sinks=4, dtype="bf16", quantised=True),
        # ragged chunks packed one behind the other, the buffer's last rows unused
        dict(name="window odd chunks", op="window", batch=5, new=1003, heads=20, kv_heads=4, dim=96, page=16, shortest=700, longest=3001, window=513,
             sinks=5, dtype="f16", quantised=False),
        # a whole prompt
        dict(name="window prompt", op="window", batch=1, new=8192, heads=32, kv_heads=8, dim=128, page=64, shortest=8192, longest=8192, window=4096,
             sinks=16, dtype="bf16", quantised=False),
        # a chunk of each of a few prompts that see everything before it, in an 8-bit cache
        dict(name="whole chunk", op="window", batch=4, new=512, heads=32, kv_heads=8, dim=128, page=16, shortest=2100, longest=8000, window=0,
             sinks=0, dtype="bf16", quantised=True),
        # a few drafted tokens of one stream: latency
        dict(name="tree short", op="tree", batch=1, drafts=7, heads=8, kv_heads=2, dim=64, page=16, shortest=100, longest=100, dtype="bf16",
             quantised=False),
        # 16 streams of ragged lengths, an odd tree each, over an 8-bit cache
        dict(name="tree batch", op="tree", batch=16, drafts=25, heads=32, kv_heads=8, dim=128, page=16, shortest=1, longest=4096, dtype="bf16",
             quantised=True),
        # the largest usual tree over a long context: work has to be split over the length
        dict(name="tree long", op="tree", batch=2, drafts=64, heads=32, kv_heads=8, dim=128, page=64, shortest=100001, longest=131072, dtype="bf16",
             quantised=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "window", "window", "window", "tree", "tree"])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        dim = rng.choice([32, 64, 80, 96, 128])
        kv = rng.choice([1, 2, 4, 8])
        tokens = _log(rng, 1, 32768)
        return dict(op=op, tokens=tokens, heads=kv * rng.choice([1, 2, 3, 4]), kv_heads=kv, dim=dim, rotary=dim if rng.random() < 0.6 else dim // 2,
                    interleaved=rng.random() < 0.4, page=page, pages=-(-tokens // page) + rng.randrange(64), first=_log(rng, 1, 1000000) - 1,
                    dtype=rng.choice(["bf16", "f16", "f32"]), quantised=rng.random() < 0.6)
    kv, share, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 96, 128, 256])
    common = dict(heads=kv * share, kv_heads=kv, dim=dim, page=page, dtype=rng.choice(["bf16", "f16"]), quantised=rng.random() < 0.5)
    # scores of all query heads, by the work of one of them, and cache cells
    scores, cells = 3 * 2 ** 28 // (kv * share) * 128 // max(128, dim), 2 ** 28 // (kv * dim)
    if op == "window":
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, min(8192, 32768 // batch, math.isqrt(scores // batch)))
        longest = max(new, _log(rng, 1, min(131072, cells // batch)))
        reach = max(1, scores // (batch * new) - new)
        window = _log(rng, 1, min(longest, reach)) if longest > reach or rng.random() < 0.75 else 0
        return dict(op=op, batch=batch, new=new, shortest=rng.randrange(longest + 1), longest=longest, window=window,
                    sinks=rng.choice([0, 1, 4, 64, 100]) if window else 0, **common)
    batch, drafts = _log(rng, 1, 16), _log(rng, 1, 128)
    longest = _log(rng, 1, min(131072, cells // batch, scores // (batch * drafts)))
    return dict(op=op, batch=batch, drafts=drafts, shortest=rng.randrange(longest + 1), longest=longest, **common)


def _lengths(c):
    """The streams' lengths, evenly from the longest to the shortest: the case alone fixes them."""
    b, lo, hi = c["batch"], c["shortest"], c["longest"]
    return [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]


def _new(c):
    """The streams' new tokens: all of `new` where it is 1 or there is one stream, else fewer from stream to stream, at most a stream's length."""
    return [min(c["new"] - c["new"] // 2 * i // max(1, c["batch"] - 1), n) for i, n in enumerate(_lengths(c))]


def _rows(c):
    """Rows of q: the new tokens of all streams, some unused ones behind them where a stream can have several."""
    return sum(_new(c)) + (3 if c["new"] > 1 and c["batch"] > 1 else 0)


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

    def cache(pages):
        shape = (pages, c["kv_heads"], c["page"], c["dim"])
        for name in ("k", "v"):
            if c["quantised"]:
                s[name + "_cache"], s[name + "_scale"] = _quantise(randn(*shape))
            else:
                s[name + "_cache"], s[name + "_scale"] = randn(*shape).to(t), None

    s = dict(op=c["op"])
    if c["op"] == "append":
        cache(c["pages"])
        tokens = torch.arange(c["tokens"], device=DEV)
        # pages are scattered, the tokens of a page follow each other; few tokens are of as many streams
        if c["tokens"] <= 256:
            s["slots"] = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:c["tokens"]]
            s["positions"] = c["first"] + torch.randint(0, 1 + c["first"] // 2, (c["tokens"],), generator=g, device=DEV)
        else:
            s["slots"] = torch.randperm(c["pages"], generator=g, device=DEV)[tokens // c["page"]] * c["page"] + tokens % c["page"]
            s["positions"] = c["first"] + tokens
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, c["rotary"], 2, device=DEV, dtype=torch.float32) / c["rotary"])
        s["interleaved"] = c["interleaved"]
        # the three parts of one projection's output
        qkv = randn(c["tokens"], c["heads"] + 2 * c["kv_heads"], c["dim"]).to(t)
        s["q"], s["k"], s["v"] = qkv.split([c["heads"], c["kv_heads"], c["kv_heads"]], dim=1)
        return s
    lengths = torch.tensor(_lengths(c), dtype=torch.int32)
    held = c["longest"] + (c["drafts"] if c["op"] == "tree" else 0)
    width = max(1, -(-held // c["page"]))
    s["page_table"] = torch.randperm(c["batch"] * width, generator=g, device=DEV).to(torch.int32).view(c["batch"], width)
    cache(c["batch"] * width)
    s["lengths"] = lengths.to(DEV)
    s["scale"] = c["dim"] ** -0.5
    if c["op"] == "window":
        # ends of the streams' rows, in the order of the streams
        s["starts"] = torch.tensor([0] + _new(c), dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV) if _new(c) != [1] * c["batch"] else None
        s["window"], s["sinks"], s["new"] = c["window"] or None, c["sinks"], c["new"]
        s["q"] = (2 * randn(_rows(c), c["heads"], c["dim"])).to(t)
        # rows behind the last stream's stay as they are
        s["out"] = torch.zeros_like(s["q"])
        return s
    # a random tree: a draft's parent is one of those before it, or the last token of the context
    parents = (torch.rand(c["batch"], c["drafts"], generator=g, device=DEV) * (torch.arange(c["drafts"], device=DEV) + 1)).long() - 1
    sees = torch.zeros(c["batch"], c["drafts"], c["drafts"] + 1, dtype=torch.bool, device=DEV)
    for i in range(c["drafts"]):
        sees[:, i] = sees[:, i].scatter(1, parents[:, i:i + 1] % (c["drafts"] + 1), True)
        sees[:, i] |= torch.where(parents[:, i:i + 1] >= 0, sees.gather(1, parents[:, i].clamp(min=0).view(-1, 1, 1).expand(-1, 1, c["drafts"] + 1))[:, 0], False)
        sees[:, i, i] = True
    words = -(-c["drafts"] // 64)
    bits = torch.zeros(c["batch"], c["drafts"], words * 64, dtype=torch.bool, device=DEV)
    bits[:, :, :c["drafts"]] = sees[:, :, :c["drafts"]]
    weight = torch.ones(64, dtype=torch.int64, device=DEV) << torch.arange(64, device=DEV)
    s["tree"] = (bits.view(c["batch"], c["drafts"], words, 64) * weight).sum(-1)
    s["q"] = (2 * randn(c["batch"], c["drafts"], c["heads"], c["dim"])).to(t)
    return s


def _cache(s):
    """The framework's handle of a cache, kept in the state as a program keeps it."""
    if "cache" not in s:
        import convt_forward_amd as C
        s["cache"] = C.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s["cache"]


def _own(s):
    import convt_forward_amd as C
    if s["op"] == "append":
        q = C.cache_append(_cache(s), s["k"], s["v"], s["slots"], s["positions"], s["inv_freq"], q=s["q"], interleaved=s["interleaved"])
        return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if s["op"] == "window":
        return C.window_attention(s["q"], _cache(s), s["page_table"], s["lengths"], starts=s["starts"], window=s["window"], sinks=s["sinks"],
                                  scale=s["scale"], out=s["out"])
    return C.tree_attention(s["q"], _cache(s), s["page_table"], s["lengths"], s["tree"], scale=s["scale"])


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, dim] with its first 2 * cos.shape[1] dims rotated, in float32."""
    half = cos.shape[1]
    x, rest = x[..., :2 * half].float(), x[..., 2 * half:].float()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    c, s = cos.unsqueeze(1), sin.unsqueeze(1)
    pair = (a * c - b * s, a * s + b * c)
    turned = torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1)
    return torch.cat([turned, rest], -1)


def _plain_append(s):
    angle = s["positions"].double().unsqueeze(1) * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    page = s["k_cache"].shape[2]
    at, off = s["slots"] // page, s["slots"] % page

    def write(name, x):
        if s[name + "_scale"] is not None:
            x, scale = _quantise(x)
            s[name + "_scale"][at, :, off] = scale
            s[name + "_cache"].view(torch.uint8)[at, :, off] = x.view(torch.uint8)
        else:
            s[name + "_cache"][at, :, off] = x.to(s["q"].dtype)

    write("k", _rotate(s["k"], cos, sin, s["interleaved"]))
    write("v", s["v"].float())
    q = _rotate(s["q"], cos, sin, s["interleaved"]).to(s["q"].dtype)
    return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _cells(s, name, at):
    """Keys or values of the tokens `at` [batch, n] of each stream as float32 [batch, kv_heads, n, dim]."""
    page = s["k_cache"].shape[2]
    pages = s["page_table"].long().gather(1, at // page)
    if s[name + "_scale"] is None:
        return s[name + "_cache"][pages, :, at % page].transpose(1, 2).float()
    x = s[name + "_cache"].view(torch.uint8)[pages, :, at % page].view(E4M3).float()
    return (x * s[name + "_scale"][pages, :, at % page].unsqueeze(-1)).transpose(1, 2)


def _softmax_product(s, q, at, seen):
    """q [batch, n, heads, dim] over the tokens `at` [batch, m]; seen [batch, n, m]. Rows that see nothing are 0."""
    batch, n, heads, dim = q.shape
    kv = s["k_cache"].shape[1]
    q = (q.float() * s["scale"]).view(batch, n, kv, heads // kv, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv, -1, dim)
    score = torch.matmul(q, _cells(s, "k", at).transpose(-1, -2).contiguous()).view(batch, heads, n, -1)
    score.masked_fill_(~seen.unsqueeze(1), -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top.isinf(), 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(batch, kv, -1, score.shape[-1]), _cells(s, "v", at)).view(batch, heads, n, dim)
    return (out / torch.where(total > 0, total, 1.0)).transpose(1, 2)


def _plain_window(s):
    rows, batch = s["q"].shape[0], s["lengths"].shape[0]
    held = s["page_table"].shape[1] * s["k_cache"].shape[2]
    length = s["lengths"].long().unsqueeze(1)
    most = s["new"]  # of any stream
    if s["starts"] is None:
        first = torch.arange(batch, device=DEV).unsqueeze(1)
        count = torch.ones_like(first)
    else:
        first, count = s["starts"][:-1].long().unsqueeze(1), s["starts"].long().diff().unsqueeze(1)
    each = torch.arange(most, device=DEV)
    row = (first + each).clamp(max=rows - 1)
    position = length - count + each
    reach = min(held, most + (s["window"] or held))
    behind = length - reach + torch.arange(reach, device=DEV)
    at = torch.cat([torch.arange(s["sinks"], device=DEV).expand(batch, -1), behind], 1)
    # a first token that the window's part holds as well counts there
    real = torch.cat([(torch.arange(s["sinks"], device=DEV) < behind[:, :1]), behind >= 0], 1)
    p, t = position.unsqueeze(2), at.unsqueeze(1)
    near = t < s["sinks"] if s["window"] is None else (t > p - s["window"]) | (t < s["sinks"])
    seen = real.unsqueeze(1) & (t <= p) & (near if s["window"] is not None else True)
    out = _softmax_product(s, s["q"][row], at.clamp(0, held - 1), seen).to(s["q"].dtype)
    # rows past a stream's own go to a spare row
    place = torch.where(each < count, row, rows)
    full = torch.cat([s["out"], s["out"].new_empty(1, *s["out"].shape[1:])])
    full[place.flatten()] = out.flatten(0, 1)
    s["out"].copy_(full[:rows])
    return s["out"]


def _plain_tree(s):
    batch, drafts = s["q"].shape[:2]
    held = s["page_table"].shape[1] * s["k_cache"].shape[2]
    length = s["lengths"].long().view(batch, 1, 1)
    at = torch.arange(held, device=DEV).expand(batch, -1)
    j = at.unsqueeze(1) - length
    inside = (j >= 0) & (j < drafts)
    j = j.clamp(0, drafts - 1).expand(-1, drafts, -1)
    seen = (at.unsqueeze(1) < length) | (inside & (s["tree"].gather(2, j // 64) >> j % 64 & 1).bool())
    return _softmax_product(s, s["q"], at, seen).to(s["q"].dtype)


PLAIN = {"append": _plain_append, "window": _plain_window, "tree": _plain_tree}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


def _seen_window(c):
    """Keys that the rows of each stream see in all, and those that any row of it sees."""
    pairs, keys = 0, 0
    for n, new in zip(_lengths(c), _new(c)):
        window = c["window"] or n
        for p in range(n - new, n):
            lo = max(0, p - window + 1)
            pairs += p - lo + 1 + min(lo, c["sinks"])
        if new:
            lo = max(0, n - new - window + 1)
            keys += n - lo + min(lo, c["sinks"])
    return pairs, keys


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}[c["dtype"]]
    cell = c["dim"] + 4 if c["quantised"] else c["dim"] * size
    if c["op"] == "append":
        rows = c["tokens"] * (c["heads"] + c["kv_heads"])
        return {"bytes": c["tokens"] * (2 * (c["heads"] + c["kv_heads"]) * c["dim"] * size + 2 * c["kv_heads"] * cell + 16) + 2 * c["rotary"],
                "flops": 3 * rows * c["rotary"] + (6 * c["tokens"] * c["kv_heads"] * c["dim"] if c["quantised"] else 0)}
    if c["op"] == "window":
        pairs, keys = _seen_window(c)
        rows = sum(_new(c))
        extra = 8 * c["batch"]
    else:
        rows, keys = c["batch"] * c["drafts"], sum(_lengths(c)) + c["batch"] * c["drafts"]
        pairs = sum(_lengths(c)) * c["drafts"] + c["batch"] * c["drafts"]  # of the tree: at least each draft itself
        extra = 4 * c["batch"] + 8 * rows * -(-c["drafts"] // 64)
    return {"bytes": 2 * keys * c["kv_heads"] * cell + 2 * rows * c["heads"] * c["dim"] * size + 4 * -(-keys // c["page"]) + extra,
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# In 64 bits. Values held in e4m3 are given before their rounding: the error of both sides
# is then the format's own.


def _exact_append(c, s):
    heads, half = c["kv_heads"], c["rotary"] // 2
    turn = s["positions"].double()[:, None, None] * s["inv_freq"].double()

    def rotate(x):
        x = x.double().clone()
        i = torch.arange(half, device=DEV)
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(turn), turn)
        x[..., first], x[..., second] = z.real, z.imag
        return x

    found, scales = [], []
    for name, new in (("k", rotate(s["k"])), ("v", s["v"].double())):
        flat = s[name + "_cache"].double().permute(0, 2, 1, 3).reshape(-1, heads, c["dim"])
        if c["quantised"]:
            step = torch.clamp(new.abs().max(dim=-1).values / 448, min=2.0 ** -126)
            new = new / step[..., None]
            old = s[name + "_scale"].double().permute(0, 2, 1).reshape(-1, heads).index_copy(0, s["slots"], step)
            scales.append(old.view(c["pages"], c["page"], heads).permute(0, 2, 1).contiguous())
        else:
            scales.append(None)
        found.append(flat.index_copy(0, s["slots"], new).view(c["pages"], c["page"], heads, c["dim"]).permute(0, 2, 1, 3).contiguous())
    return (rotate(s["q"]), *found, *scales)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    share, done = c["heads"] // c["kv_heads"], 0
    for b, n in enumerate(_lengths(c)):
        if c["op"] == "tree":
            rows, total = s["q"][b], n + c["drafts"]
            words = s["tree"][b].tolist()
            sees = torch.tensor([[w[j // 64] >> (j % 64) & 1 for j in range(c["drafts"])] for w in words], dtype=torch.bool, device=DEV)
            hidden = torch.cat([torch.zeros(c["drafts"], n, dtype=torch.bool, device=DEV), ~sees], 1)
            into = out[b]
        else:
            new = _new(c)[b]
            rows, total = s["q"][done:done + new], n
            into = out[done:done + new]
            done += new
            if new == 0:
                continue
            p = torch.arange(n - new, n, device=DEV)[:, None]
            t = torch.arange(n, device=DEV)
            hidden = (t > p) | ((t + (c["window"] or n) <= p) & (t >= c["sinks"]))
        pages = s["page_table"][b, :-(-total // c["page"])].long()
        for h in range(c["kv_heads"]):
            kv = []
            for name in ("k", "v"):
                x = s[name + "_cache"][:, h]
                x = x.view(torch.uint8)[pages].view(E4M3) if c["quantised"] else x[pages]
                x = x.double() * (s[name + "_scale"][:, h][pages].double()[..., None] if c["quantised"] else 1)
                kv.append(x.reshape(-1, c["dim"])[:total])
            for i in range(h * share, (h + 1) * share):
                score = (rows[:, i].double() @ kv[0].t()) * s["scale"]
                into[:, i] = torch.softmax(score.masked_fill_(hidden, -math.inf), dim=1) @ kv[1]
    return out
