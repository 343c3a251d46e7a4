"""The operators of libconvt for steps with several new tokens per stream (include/convt_extend.h)
on torch tensors: prompts and chunks of them, long streams that see a window, trees of drafted tokens.

    q = convt_forward_amd.cache_append(cache, k, v, slots, positions, inv_freq, q=q)
    out = convt_forward_amd.window_attention(q, cache, page_table, lengths, starts, window=4096, sinks=4)
    out = convt_forward_amd.tree_attention(q, cache, page_table, lengths, convt_forward_amd.tree_mask(parents))

They stand beside cache_write and decode_attention and work on the same KVCache, with the same
conventions: device tensors, outputs and workspaces allocated with torch when not given, calls
enqueued on torch's current stream or on `stream`, ValueError or ConvtError for wrong arguments,
no fallback, no gradients.
"""
from __future__ import annotations

import ctypes
import math
import operator
from typing import Optional, Tuple

import torch

from . import _on_device, _tie_to_stream
from . import lib as _load
from .decode import (CacheDesc, CacheRows, KVCache, _cache_rows, _check, _check_workspace, _empty, _f32, _i32, _i64,
                     _launch_stream, _ptr, _raise, _vp)

EXTEND_ROUTES = {"auto": 0, "direct": 1, "mfma": 2}


class AppendProblem(ctypes.Structure):
    _fields_ = [("cache", CacheDesc), ("rows", CacheRows), ("q_stride", _i64 * 2), ("q_out_stride", _i64 * 2), ("heads", _i32),
                ("rotary_dim", _i32), ("interleaved", _i32), ("reserved", _i32)]


class WindowProblem(ctypes.Structure):
    _fields_ = [("cache", CacheDesc), ("max_length", _i64), ("tokens", _i64), ("q_stride", _i64 * 2), ("out_stride", _i64 * 2),
                ("table_width", _i64), ("table_stride", _i64), ("window", _i64), ("sinks", _i64), ("batch", _i32),
                ("heads", _i32), ("ragged", _i32), ("route", _i32), ("scale", _f32), ("reserved", _i32)]


class TreeProblem(ctypes.Structure):
    _fields_ = [("cache", CacheDesc), ("max_length", _i64), ("q_stride", _i64 * 3), ("out_stride", _i64 * 3),
                ("tree_stride", _i64 * 2), ("table_width", _i64), ("table_stride", _i64), ("batch", _i32), ("drafts", _i32),
                ("heads", _i32), ("route", _i32), ("scale", _f32), ("reserved", _i32)]


class ExtendInfo(ctypes.Structure):
    _fields_ = [("workspace_bytes", _i64), ("route", _i32), ("chunks", _i32), ("chunk_tokens", _i32), ("reserved", _i32)]


_ready = None


def lib() -> ctypes.CDLL:
    """libconvt.so with the entry points of this module declared."""
    global _ready
    if _ready is None:
        L = _load()
        P = ctypes.POINTER
        for name, args in {
            "convt_cache_append": [P(AppendProblem)] + [_vp] * 12,
            "convt_window_query": [P(WindowProblem), P(ExtendInfo)],
            "convt_window_attend": [P(WindowProblem)] + [_vp] * 12,
            "convt_tree_query": [P(TreeProblem), P(ExtendInfo)],
            "convt_tree_attend": [P(TreeProblem)] + [_vp] * 12,
        }.items():
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_int
        _ready = L
    return _ready


def _vector(t, name: str, shape, dtype, device) -> None:
    """A contiguous vector of its own shape and type."""
    _check(t, name, shape, dtype, device)
    if shape[0] > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


def _form(t):
    """What a call's checks and its problem know of a tensor."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _append_problem(cache: KVCache, k, v, slots, positions, inv_freq, q, interleaved, q_out) -> AppendProblem:
    rows = _cache_rows(cache, k, v, slots)
    tokens, dim, device = rows.tokens, cache.head_dim, cache.device
    d = cache._desc(k.dtype, "k")
    _vector(positions, "positions", (tokens,), torch.int64, device)
    if inv_freq.dim() != 1 or 2 * inv_freq.shape[0] > dim:
        raise ValueError(f"inv_freq must have one axis of at most {dim // 2} entries")
    half = inv_freq.shape[0]
    _vector(inv_freq, "inv_freq", (half,), torch.float32, device)
    heads, strides = 0, [(0, 0)] * 2
    if q is not None:
        if q.dim() != 3 or q.shape[0] != tokens or q.shape[2] != dim:
            raise ValueError(f"q must be [{tokens}, heads, {dim}]")
        _check(q, "q", None, k.dtype, device)
        heads = _count(q.shape[1], "heads")
        if heads == 0:
            raise ValueError("q has no heads")
        if q_out is not None:
            _check(q_out, "q_out", q.shape, q.dtype, device)
        strides = []
        for t, name in ((q, "q"), (q_out, "q_out")):
            s = (heads * dim, dim, 1) if t is None else t.stride()
            if dim > 1 and s[2] != 1:
                raise ValueError(f"the last axis of {name} must be contiguous")
            strides.append((s[0] if tokens > 1 else heads * dim, s[1] if heads > 1 else dim))
    elif q_out is not None:
        raise ValueError("q_out without q")
    return AppendProblem(d, rows, (_i64 * 2)(*strides[0]), (_i64 * 2)(*strides[1]), heads, 2 * half, 1 if interleaved else 0, 0)


def cache_append(cache: KVCache, k, v, slots, positions, inv_freq, q=None, interleaved: bool = False, q_out=None, stream=None):
    """Rotate q and k by their tokens' positions, and write k and v into the cache at slots.

    k and v [tokens, kv_heads, head_dim], q [tokens, heads, head_dim]; slots and positions int64
    [tokens]; inv_freq float32 [rotary_dim / 2], the angle a position turns pair i by: of dims
    (i, i + rotary_dim / 2), or (2i, 2i + 1) if interleaved. Dims from rotary_dim on stay. Tokens
    whose slot lies outside the cache are not written (their queries are rotated); a slot given
    twice may be left with parts of both tokens. A quantised cache takes the rotated keys per token
    and head, as cache_write does. Returns the rotated queries (q_out, which may be q), None
    without q. positions and inv_freq are float64 factors in the kernel: far positions keep their
    angles."""
    # the checks and the problem follow from the tensors' forms: kept for calls of the same ones (12.6 us a
    # call without, 64 tokens)
    key = ("append", _form(k), _form(v), _form(slots), _form(positions), _form(inv_freq), _form(q), _form(q_out), bool(interleaved))
    p = cache._attends.get(key)
    if p is None:
        p = _append_problem(cache, k, v, slots, positions, inv_freq, q, interleaved, q_out)
        if len(cache._attends) >= 256:
            cache._attends.clear()
        cache._attends[key] = p
    device, owned = cache.device, []
    sh, ext = _launch_stream(stream, device)
    if q is not None and q_out is None:
        q_out = _empty(q.shape, q.dtype, device)
        owned.append(q_out)
    st = _on_device(device, (_ready or lib()).convt_cache_append, ctypes.byref(p), _ptr(q), k.data_ptr(), v.data_ptr(),
                    slots.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(),
                    _ptr(cache.k_scale), _ptr(cache.v_scale), _ptr(q_out), sh)
    if st:
        _raise(st, "convt_cache_append")
    if ext is not None:
        _tie_to_stream(owned, ext)
    return q_out


def tree_mask(parents):
    """The tree of tree_attention from its drafts' parents: int64 [..., drafts, (drafts + 63) // 64]
    whose bit j of row i says that draft j is i or one of its ancestors. parents [..., drafts]
    holds for each draft the draft it follows, or -1 (or any number that is no draft's) for one that
    follows the cached tokens; drafts may come in any order. Plain torch, on parents' device."""
    drafts = parents.shape[-1]
    parents = parents.to(torch.int64)
    # an index out of range would end the process where parents are on a device
    parents = torch.where(parents < drafts, parents, -1)
    words = (drafts + 63) // 64
    at = torch.arange(drafts, device=parents.device)
    rows = torch.zeros(parents.shape + (words,), dtype=torch.int64, device=parents.device)
    rows.scatter_(-1, (at // 64).expand(parents.shape).unsqueeze(-1),
                  torch.ones_like(at).bitwise_left_shift(at % 64).expand(parents.shape).unsqueeze(-1))
    # after a turn a row holds twice as many generations, and `parents` are that far up
    for _ in range((drafts - 1).bit_length()):
        up = parents.clamp(min=0)
        theirs = rows.gather(-2, up.unsqueeze(-1).expand(rows.shape))
        rows = rows | torch.where((parents >= 0).unsqueeze(-1), theirs, 0)
        parents = torch.where(parents >= 0, parents.gather(-1, up), -1)
    return rows


def _number(scale):
    # plain numbers: a tensor in a plan's key would stand for itself, not for its value
    return None if scale is None else float(scale)


_LIMIT = 2 ** 62  # numbers beyond it mean no other thing than this; ctypes would cut them to 64 bits


def _index(value):
    return None if value is None else max(-_LIMIT, min(operator.index(value), _LIMIT))


def _count(value: int, name: str) -> int:
    """A size that a problem holds in 32 bits, to which ctypes would cut it."""
    if value >= 2 ** 31:
        raise ValueError(f"more than 2^31 - 1 {name}")
    return value


def _check_query(cache: KVCache, q, page_table, ragged: bool, out, axes: str) -> None:
    """q and out have the axes; a page table has a row for each entry of q's first one, unless ragged."""
    if q.dim() != axes.count(",") + 1 or q.shape[-1] != cache.head_dim:
        raise ValueError(f"q must be [{axes[:-3]}{cache.head_dim}]")
    if page_table.dim() != 2 or not (ragged or page_table.shape[0] == q.shape[0]):
        raise ValueError(f"page_table must be [{'batch' if ragged else q.shape[0]}, pages]")
    for t, name in ((q, "q"), (out, "out")):
        if t is not None and cache.head_dim > 1 and t.stride(-1) != 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("the last axis of page_table must be contiguous")


def _strides(shape, stride):
    """All but the last stride; an axis of one entry (or none) has none of its own."""
    packed, n = [], 1
    for v in reversed(shape):
        packed.append(n)
        n *= max(1, v)
    return (_i64 * (len(shape) - 1))(*(s if v > 1 else c for v, s, c in zip(shape[:-1], stride, packed[::-1])))


def _plan(cache: KVCache, key, make, query: str):
    """The problem that make() gives and its info, kept with the cache for calls of the same shapes."""
    got = cache._attends.get(key)
    if got is None:
        p, info = make(), ExtendInfo()
        st = getattr(_ready or lib(), query)(ctypes.byref(p), ctypes.byref(info))
        if st:
            _raise(st, query)
        if len(cache._attends) >= 256:
            cache._attends.clear()
        got = cache._attends[key] = (p, info)
    return got


def window_plan(cache: KVCache, q, page_table, ragged: bool = False, window: Optional[int] = None, sinks: int = 0, scale=None,
                max_length: Optional[int] = None, out=None, route: str = "auto") -> Tuple[WindowProblem, ExtendInfo]:
    """The problem and the route, parts and workspace size of a window_attention call on these
    tensors; ragged: whether starts is given."""
    scale, max_length, window, sinks = _number(scale), _index(max_length), _index(window), _index(operator.index(sinks))
    out_stride = None if out is None else out.stride()
    key = ("window", q.dtype, q.shape, q.stride(), page_table.shape, page_table.stride(), bool(ragged), window, sinks, scale, max_length,
           out_stride, route)

    def make():
        if window is not None and window < 1:
            raise ValueError("window must be at least 1 (None: everything before a token)")
        _check_query(cache, q, page_table, ragged, out, "tokens, heads, dim")
        batch, width = page_table.shape
        tokens, heads, dim = q.shape
        return WindowProblem(cache._desc(q.dtype, "q"), width * cache.page_size if max_length is None else max_length, tokens,
                             _strides(q.shape, q.stride()), _strides(q.shape, out_stride or (heads * dim, dim, 1)), width,
                             page_table.stride(0) if batch > 1 else max(1, width), window or 0, sinks,
                             _count(batch, "streams"), _count(heads, "heads"), 1 if ragged else 0, EXTEND_ROUTES[route],
                             1.0 / math.sqrt(dim) if scale is None else scale, 0)

    return _plan(cache, key, make, "convt_window_query")


def _finish(cache, q, info, out, lse, workspace, lse_shape):
    """Outputs and workspace of a call, and which of them are made here."""
    owned = []
    if out is None:
        out = _empty(q.shape, q.dtype, cache.device)
        owned.append(out)
    lse_t = None
    if lse is True:
        lse_t = _empty(lse_shape, torch.float32, cache.device)
        owned.append(lse_t)
    elif lse is not False and lse is not None:
        _check(lse, "lse", lse_shape, torch.float32, cache.device)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        lse_t = lse
    if workspace is None:
        if info.workspace_bytes:
            workspace = _empty((info.workspace_bytes,), torch.uint8, cache.device)
            owned.append(workspace)
    else:
        _check_workspace(workspace, info.workspace_bytes, cache.device)
    return out, lse_t, workspace, owned


def window_attention(q, cache: KVCache, page_table, lengths, starts=None, window: Optional[int] = None, sinks: int = 0,
                     scale: Optional[float] = None, max_length: Optional[int] = None, out=None, lse=False, workspace=None,
                     stream=None, route: str = "auto"):
    """Causal attention of the streams' new tokens over their cached ones, with a window and
    first tokens that stay visible.

    q [tokens, heads, head_dim] holds the new tokens of all streams: rows starts[b] to
    starts[b + 1] (int32 [batch + 1], not decreasing) are the last ones of the lengths[b]
    tokens of stream b (int32 [batch]), all in the cache; without starts every stream has one. A
    token at position p sees the tokens t <= p with t > p - window or t < sinks (all t <= p
    without a window). page_table int32 [batch, pages]; heads / kv_heads query heads share a kv
    head; scale is 1 / sqrt(head_dim) by default. max_length bounds the lengths (default: what
    the table can hold). A given workspace is contiguous, with at least window_plan's
    workspace_bytes. Returns out [tokens, heads, head_dim]; with lse (True, or a float32 tensor
    [tokens, heads] to fill) the pair (out, lse). A row that sees nothing gets zeros and
    -infinity. Rows behind the last stream's are not written. On the matrix cores weights are rounded
    to 11 bits over float16 and e4m3 caches, and over bfloat16 ones to 8, or 16 in calls of few rows
    (convt_extend.h has the rule); route="direct" keeps float32."""
    _check(q, "q", None, None, cache.device)
    _check(page_table, "page_table", None, torch.int32, cache.device)
    if out is not None:
        _check(out, "out", q.shape, q.dtype, cache.device)
    p, info = window_plan(cache, q, page_table, starts is not None, window, sinks, scale, max_length, out, route)
    _vector(lengths, "lengths", (p.batch,), torch.int32, cache.device)
    if starts is not None:
        _vector(starts, "starts", (p.batch + 1,), torch.int32, cache.device)
    sh, ext = _launch_stream(stream, cache.device)
    out, lse_t, workspace, owned = _finish(cache, q, info, out, lse, workspace, q.shape[:2])
    st = _on_device(cache.device, (_ready or lib()).convt_window_attend, ctypes.byref(p), q.data_ptr(), cache.k.data_ptr(),
                    cache.v.data_ptr(), _ptr(cache.k_scale), _ptr(cache.v_scale), page_table.data_ptr(), lengths.data_ptr(),
                    _ptr(starts), out.data_ptr(), _ptr(lse_t), _ptr(workspace), sh)
    if st:
        _raise(st, "convt_window_attend")
    if ext is not None:
        _tie_to_stream(owned, ext)
    return out if lse_t is None else (out, lse_t)


def tree_plan(cache: KVCache, q, page_table, tree, scale=None, max_length: Optional[int] = None, out=None,
              route: str = "auto") -> Tuple[TreeProblem, ExtendInfo]:
    """The problem and the route, parts and workspace size of a tree_attention call on these tensors."""
    scale, max_length = _number(scale), _index(max_length)
    out_stride = None if out is None else out.stride()
    key = ("tree", q.dtype, q.shape, q.stride(), page_table.shape, page_table.stride(), tree.shape, tree.stride(), scale, max_length,
           out_stride, route)

    def make():
        _check_query(cache, q, page_table, False, out, "batch, drafts, heads, dim")
        batch, drafts, heads, dim = q.shape
        words = (drafts + 63) // 64
        if tree.shape != (batch, drafts, words) and tree.shape != (drafts, words):
            raise ValueError(f"tree must be [{batch}, {drafts}, {words}] or [{drafts}, {words}]")
        if words > 1 and tree.stride(-1) != 1:
            raise ValueError("the last axis of tree must be contiguous")
        width = page_table.shape[1]
        tree_stride = (_i64 * 2)(tree.stride(0) if tree.dim() == 3 and batch > 1 else 0, tree.stride(-2) if drafts > 1 else words)
        return TreeProblem(cache._desc(q.dtype, "q"), width * cache.page_size if max_length is None else max_length,
                           _strides(q.shape, q.stride()), _strides(q.shape, out_stride or (drafts * heads * dim, heads * dim, dim, 1)),
                           tree_stride, width, page_table.stride(0) if batch > 1 else max(1, width), _count(batch, "streams"),
                           _count(drafts, "drafts"), _count(heads, "heads"), EXTEND_ROUTES[route], 1.0 / math.sqrt(dim) if scale is None else scale, 0)

    return _plan(cache, key, make, "convt_tree_query")


def tree_attention(q, cache: KVCache, page_table, lengths, tree, scale: Optional[float] = None, max_length: Optional[int] = None,
                   out=None, lse=False, workspace=None, stream=None, route: str = "auto"):
    """Attention of drafted tokens over their stream's cached tokens and over each other.

    q [batch, drafts, heads, head_dim]; lengths int32 [batch], the tokens before the drafts, which
    every draft sees; the cache holds draft j of stream b at position lengths[b] + j of its page
    table (its key rotated for its own position, that of its depth). tree int64 [batch, drafts, (drafts +
    63) // 64], or without the batch where all streams have the same: draft i sees draft j if bit
    j % 64 of tree[b, i, j // 64] is set (tree_mask makes it from the drafts' parents).
    page_table int32 [batch, pages]; heads / kv_heads query heads share a kv head; scale is 1 /
    sqrt(head_dim) by default. max_length bounds the cached tokens, the drafts among them (default: what
    the table can hold); those past it are left out. A given workspace is contiguous, with at
    least tree_plan's workspace_bytes. Returns out, of q's shape; with lse (True, or a float32
    tensor [batch, drafts, heads] to fill) the pair (out, lse). A draft that sees nothing gets
    zeros and -infinity."""
    _check(q, "q", None, None, cache.device)
    _check(page_table, "page_table", None, torch.int32, cache.device)
    _check(tree, "tree", None, torch.int64, cache.device)
    if out is not None:
        _check(out, "out", q.shape, q.dtype, cache.device)
    p, info = tree_plan(cache, q, page_table, tree, scale, max_length, out, route)
    _vector(lengths, "lengths", (p.batch,), torch.int32, cache.device)
    sh, ext = _launch_stream(stream, cache.device)
    out, lse_t, workspace, owned = _finish(cache, q, info, out, lse, workspace, q.shape[:3])
    st = _on_device(cache.device, (_ready or lib()).convt_tree_attend, ctypes.byref(p), q.data_ptr(), cache.k.data_ptr(),
                    cache.v.data_ptr(), _ptr(cache.k_scale), _ptr(cache.v_scale), page_table.data_ptr(), lengths.data_ptr(),
                    tree.data_ptr(), out.data_ptr(), _ptr(lse_t), _ptr(workspace), sh)
    if st:
        _raise(st, "convt_tree_attend")
    if ext is not None:
        _tie_to_stream(owned, ext)
    return out if lse_t is None else (out, lse_t)
