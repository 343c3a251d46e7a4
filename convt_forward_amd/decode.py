"""The decoding-step operators of libconvt (include/convt_decode.h) on torch tensors.

    cache = convt_forward_amd.KVCache.new(n_pages, kv_heads, page_size, head_dim, quantised=True)
    y, y_scale, h = convt_forward_amd.rms_norm(x, weight, residual=h, quantise=True)
    qkv = convt_forward_amd.q4_matvec(y, w, w_scales, x_scale=y_scale)
    convt_forward_amd.cache_write(cache, k, v, slots)
    out = convt_forward_amd.decode_attention(q, cache, page_table, lengths)

As in the rest of the package, Python only marshals arguments: tensors are
device tensors, outputs and workspaces are allocated with torch when not
given, calls are enqueued on torch's current stream or on `stream`, wrong
arguments raise ValueError (from here) or ConvtError (from the library), and
nothing falls back to another implementation. None of these calls is
differentiable: they serve inference.
"""
from __future__ import annotations

import ctypes
import math
import operator
from typing import Dict, Optional, Tuple

import torch

from . import ConvtError, DTYPES, _launch_stream as _given_stream, _on_device, _tie_to_stream
from . import lib as _load

ATTEND_ROUTES = {"auto": 0, "direct": 1, "mfma": 2}
Q4_ROUTES = {"auto": 0, "direct": 1, "mfma": 2}

_CODES = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"], torch.float16: DTYPES["f16"]}
_E4M3 = torch.float8_e4m3fn

_i64, _i32, _f32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", _i64), ("width", _i64), ("x_stride", _i64), ("residual_stride", _i64), ("y_stride", _i64),
                ("residual_out_stride", _i64), ("dtype", _i32), ("has_residual", _i32), ("quantise", _i32),
                ("eps", _f32)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("n_pages", _i64), ("k_stride", _i64 * 3), ("v_stride", _i64 * 3), ("kv_heads", _i32),
                ("page_size", _i32), ("head_dim", _i32), ("dtype", _i32), ("quantised", _i32), ("reserved", _i32)]


class CacheRows(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("k_stride", _i64 * 2), ("v_stride", _i64 * 2)]


class AttendProblem(ctypes.Structure):
    _fields_ = [("cache", CacheDesc), ("max_length", _i64), ("q_stride", _i64 * 2), ("out_stride", _i64 * 2),
                ("table_width", _i64), ("table_stride", _i64), ("batch", _i32), ("heads", _i32), ("route", _i32),
                ("scale", _f32)]


class AttendInfo(ctypes.Structure):
    _fields_ = [("workspace_bytes", _i64), ("route", _i32), ("chunks", _i32), ("chunk_tokens", _i32),
                ("reserved", _i32)]


class Q4Problem(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n", _i64), ("k", _i64), ("group", _i64), ("x_stride", _i64), ("y_stride", _i64),
                ("dtype", _i32), ("x_quantised", _i32), ("route", _i32), ("reserved", _i32)]


_ready = None


def lib() -> ctypes.CDLL:
    """libconvt.so with the decoding-step entry points declared."""
    global _ready
    if _ready is None:
        L = _load()
        P = ctypes.POINTER
        for name, args in {
            "convt_rms_norm": [P(NormProblem)] + [_vp] * 7,
            "convt_cache_write": [P(CacheDesc), P(CacheRows)] + [_vp] * 8,
            "convt_cache_read": [P(CacheDesc), P(CacheRows)] + [_vp] * 8,
            "convt_attend_query": [P(AttendProblem), P(AttendInfo)],
            "convt_attend": [P(AttendProblem)] + [_vp] * 11,
            "convt_q4_query": [P(Q4Problem), P(_i32)],
            "convt_q4_matvec": [P(Q4Problem)] + [_vp] * 6,
        }.items():
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_int
        _ready = L
    return _ready


def _raise(st: int, name: str) -> None:
    raise ConvtError(st, name)


def _launch_stream(stream, device):
    """_launch_stream of the package; the current stream's handle without making a Stream
    object, which costs as much as the launch itself."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index), None
    return _given_stream(stream, device)


def _code(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    return code


def _check(t, name: str, shape=None, dtype=None, device=None) -> None:
    if device is None:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
    elif t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(t, name: str) -> Tuple[int, int]:
    """(rows, row stride) of t[..., width]: the last axis contiguous, the
    leading ones evenly spaced."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 0:
        raise ValueError(f"{name} must have at least one axis")
    width = shape[-1]
    if width > 1 and stride[-1] != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    if len(shape) == 2:
        return shape[0], stride[0]
    if 0 in shape[:-1]:
        return 0, width
    rows, step = 1, 0
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if rows == 1:
            step = s
        elif s != rows * step:
            raise ValueError(f"the leading axes of {name} are not evenly spaced: make it contiguous")
        rows *= n
    return rows, step if rows > 1 else width


def _empty(shape, dtype, device):
    """A new contiguous tensor. empty_strided skips most of what torch.empty does with its
    arguments (1.3 against 2.1 us, a third of a small call)."""
    stride, n = [], 1
    for v in reversed(shape):
        stride.append(n)
        n *= v if v > 1 else 1
    return torch.empty_strided(shape, stride[::-1], dtype=dtype, device=device)


def _check_workspace(t, need: int, device) -> None:
    """need bytes from t's first element on are t's own (an expanded tensor has fewer than it counts)."""
    _check(t, "workspace", device=device)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if t.numel() * t.element_size() < need:
        raise ValueError("workspace too small")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def rms_norm(x, weight, residual=None, eps: float = 1e-6, quantise: bool = False, y=None, scale=None,
             residual_out=None, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight over the last axis.

    Returns (y, scale, residual_out): with `quantise`, y holds e4m3 codes
    (torch.float8_e4m3fn) and scale one float32 per row, y * scale being the
    norm; else scale is None. residual_out is h in x's type, None without a
    residual; it may be given as `residual` (or x) itself to update in place.
    x[..., width] is float32, bfloat16 or float16 with any even spacing of rows."""
    code = _code(x, "x")
    _check(x, "x")
    shape, dtype, device = x.shape, x.dtype, x.device
    rows, xs = _rows(x, "x")
    width = shape[-1]
    _check(weight, "weight", (width,), dtype, device)
    if width > 1 and weight.stride(0) != 1:
        raise ValueError("weight must be contiguous")
    sh, ext = _launch_stream(stream, device)
    owned = []
    rs = ros = 0
    if residual is not None:
        _check(residual, "residual", shape, dtype, device)
        rs = _rows(residual, "residual")[1]
        if residual_out is None:
            residual_out = _empty(shape, dtype, device)
            owned.append(residual_out)
            ros = width
        else:
            _check(residual_out, "residual_out", shape, dtype, device)
            ros = _rows(residual_out, "residual_out")[1]
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    out_dtype = _E4M3 if quantise else dtype
    if y is None:
        y = _empty(shape, out_dtype, device)
        owned.append(y)
        ys = width
    else:
        _check(y, "y", shape, out_dtype, device)
        ys = _rows(y, "y")[1]
    if quantise:
        if scale is None:
            scale = _empty(shape[:-1], torch.float32, device)
            owned.append(scale)
        else:
            _check(scale, "scale", shape[:-1], torch.float32, device)
            if not scale.is_contiguous():
                raise ValueError("scale must be contiguous")
    elif scale is not None:
        raise ValueError("scale without quantise")
    p = NormProblem(rows, width, xs, rs, ys, ros, code, 0 if residual is None else 1, 1 if quantise else 0, eps)
    st = _on_device(device, (_ready or lib()).convt_rms_norm, ctypes.byref(p), x.data_ptr(), weight.data_ptr(),
                    _ptr(residual), y.data_ptr(), _ptr(scale), _ptr(residual_out), sh)
    if st:
        _raise(st, "convt_rms_norm")
    if ext is not None:
        _tie_to_stream(owned, ext)
    return y, scale, residual_out


class KVCache:
    """A paged key-value cache: k and v [n_pages, kv_heads, page_size, head_dim] with any
    strides whose last is 1 (a [page, token, head, dim] cache is passed as its permuted view). With
    k_scale and v_scale (contiguous float32 [n_pages, kv_heads, page_size]) k and v
    hold e4m3 codes (torch.float8_e4m3fn); else they hold the element type. The tensors stay the
    caller's; one of the same shape may be put in another's place (cache.k = ...), the other
    attributes follow from them. Slot s of a page table stands for page s // page_size, token s % page_size."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4:
            raise ValueError("k must be [n_pages, kv_heads, page_size, head_dim]")
        if (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale go together")
        quantised = k_scale is not None
        if not quantised:
            _code(k, "k")
        _check(k, "k", None, _E4M3 if quantised else None)
        _check(v, "v", k.shape, k.dtype, k.device)
        n_pages, kv_heads, page_size, head_dim = k.shape
        for t, name in ((k, "k"), (v, "v")):
            if head_dim > 1 and t.stride(3) != 1:
                raise ValueError(f"the last axis of {name} must be contiguous")
        if quantised:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _check(t, name, k.shape[:3], torch.float32, k.device)
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
        # descriptions and plans of calls, which hold the tensors' strides
        descs: Dict[torch.dtype, CacheDesc] = {}
        attends: Dict[tuple, tuple] = {}
        self.__dict__.update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, quantised=quantised, n_pages=n_pages, kv_heads=kv_heads,
                             page_size=page_size, head_dim=head_dim, device=k.device, _descs=descs, _attends=attends)

    def __setattr__(self, name, value):
        if name not in ("k", "v", "k_scale", "v_scale"):
            raise AttributeError(f"{name} of a KVCache cannot be assigned")
        tensors = dict(k=self.k, v=self.v, k_scale=self.k_scale, v_scale=self.v_scale)
        tensors[name] = value
        self.__init__(**tensors)

    @classmethod
    def new(cls, n_pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=torch.bfloat16, quantised=False,
            device="cuda") -> "KVCache":
        """An empty cache of zeros, stored page by page and head by head (the order in which
        decode_attention reads it)."""
        shape = (n_pages, kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(_E4M3) if quantised else
                torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        if not quantised:
            return cls(k, v)
        return cls(k, v, *(torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))

    def _desc(self, dtype, name: str) -> CacheDesc:
        """The cache's description for rows of `dtype`."""
        d = self._descs.get(dtype)
        if d is None:
            if dtype not in _CODES:
                raise ValueError(f"{name} must be float32, bfloat16 or float16")
            if not self.quantised and dtype != self.k.dtype:
                raise ValueError(f"{name} must be {self.k.dtype}, the cache's type")
            # an axis of one entry (or none) has no stride of its own
            strides = [[t.stride(i) if t.shape[i] > 1 else max(1, self.head_dim) for i in range(3)]
                       for t in (self.k, self.v)]
            d = CacheDesc(self.n_pages, (_i64 * 3)(*strides[0]), (_i64 * 3)(*strides[1]), self.kv_heads,
                          self.page_size, self.head_dim, _CODES[dtype], 1 if self.quantised else 0, 0)
            self._descs[dtype] = d
        return d


def _cache_rows(cache: KVCache, k, v, slots) -> CacheRows:
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim) if slots.dim() == 1 else None
    if shape is None:
        raise ValueError("slots must have one axis")
    _check(slots, "slots", None, torch.int64, cache.device)
    if shape[0] > 1 and slots.stride(0) != 1:
        raise ValueError("slots must be contiguous")
    _check(k, "k", shape, None, cache.device)
    _check(v, "v", shape, k.dtype, cache.device)
    strides = []
    for t, name in ((k, "k"), (v, "v")):
        s = t.stride()
        if shape[2] > 1 and s[2] != 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
        strides.append((_i64 * 2)(s[0] if shape[0] > 1 else max(1, shape[2]), s[1] if shape[1] > 1 else max(1, shape[2])))
    return CacheRows(shape[0], *strides)


def cache_write(cache: KVCache, k, v, slots, stream=None) -> KVCache:
    """Write tokens' keys and values (k and v [tokens, kv_heads, head_dim]) into the
    cache at slots (int64 [tokens]), quantised per token and head if the cache
    is. Tokens whose slot lies outside the cache are not written; a slot given twice may be
    left with parts of both tokens. Returns the cache."""
    rows = _cache_rows(cache, k, v, slots)
    d = cache._desc(k.dtype, "k")
    sh, _ = _launch_stream(stream, cache.device)
    st = _on_device(cache.device, (_ready or lib()).convt_cache_write, ctypes.byref(d), ctypes.byref(rows), k.data_ptr(),
                    v.data_ptr(), slots.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(), _ptr(cache.k_scale),
                    _ptr(cache.v_scale), sh)
    if st:
        _raise(st, "convt_cache_write")
    return cache


def cache_read(cache: KVCache, slots, dtype=None, k=None, v=None, stream=None):
    """The keys and values at slots as (k, v), each [tokens, kv_heads, head_dim] of
    `dtype` (the cache's own type by default, bfloat16 for a quantised one); zeros
    for a slot outside the cache."""
    owned = []
    if dtype is None:
        dtype = k.dtype if k is not None else torch.bfloat16 if cache.quantised else cache.k.dtype
    d = cache._desc(dtype, "dtype")
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim) if slots.dim() == 1 else None
    if shape is None:
        raise ValueError("slots must have one axis")
    sh, ext = _launch_stream(stream, cache.device)
    if k is None:
        k = _empty(shape, dtype, cache.device)
        owned.append(k)
    if v is None:
        v = _empty(shape, dtype, cache.device)
        owned.append(v)
    if k.dtype != dtype:
        raise ValueError(f"k must be {dtype}")
    rows = _cache_rows(cache, k, v, slots)
    st = _on_device(cache.device, (_ready or lib()).convt_cache_read, ctypes.byref(d), ctypes.byref(rows),
                    cache.k.data_ptr(), cache.v.data_ptr(), _ptr(cache.k_scale), _ptr(cache.v_scale), slots.data_ptr(),
                    k.data_ptr(), v.data_ptr(), sh)
    if st:
        _raise(st, "convt_cache_read")
    if ext is not None:
        _tie_to_stream(owned, ext)
    return k, v


def cache_slots(page_table, streams, positions, page_size: int):
    """The slots (int64) of the tokens at `positions` of `streams` (rows of page_table). A
    position before the first or past what the table can hold has slot -1, which is no place of
    a cache: it is not written, and read as zeros."""
    width = page_table.shape[1]
    if width == 0:
        return torch.full_like(streams + positions, -1, dtype=torch.int64)
    at = torch.div(positions, page_size, rounding_mode="floor")
    inside = at.clamp(0, width - 1)
    slots = page_table[streams, inside].to(torch.int64) * page_size + positions % page_size
    return slots.masked_fill_(at != inside, -1)


def attend_plan(cache: KVCache, q, page_table, scale=None, max_length: Optional[int] = None, out=None,
                route: str = "auto") -> Tuple[AttendProblem, AttendInfo]:
    """The problem and the route, parts and workspace size of a decode_attention call
    on these tensors (kept with the cache for calls of the same shapes)."""
    # plain numbers: a tensor in the key would stand for itself, not for its value
    if scale is not None:
        scale = float(scale)
    if max_length is not None:
        max_length = operator.index(max_length)
    out_stride = None if out is None else out.stride()
    key = (q.dtype, q.shape, q.stride(), page_table.shape, page_table.stride(), scale, max_length, out_stride, route)
    got = cache._attends.get(key)
    if got is not None:
        return got
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError(f"q must be [batch, heads, {cache.head_dim}]")
    batch, heads, dim = q.shape
    if page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError(f"page_table must be [{batch}, pages]")
    for t, name in ((q, "q"), (out, "out")):
        if t is not None and dim > 1 and t.stride(2) != 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("the last axis of page_table must be contiguous")
    width = page_table.shape[1]

    def strides(s):
        return (_i64 * 2)(s[0] if batch > 1 else heads * dim, s[1] if heads > 1 else dim)

    p = AttendProblem(cache._desc(q.dtype, "q"), width * cache.page_size if max_length is None else max_length,
                      strides(q.stride()), strides(out_stride or (heads * dim, dim, 1)), width,
                      page_table.stride(0) if batch > 1 else max(1, width), batch, heads, ATTEND_ROUTES[route],
                      1.0 / math.sqrt(dim) if scale is None else scale)
    info = AttendInfo()
    st = (_ready or lib()).convt_attend_query(ctypes.byref(p), ctypes.byref(info))
    if st:
        _raise(st, "convt_attend_query")
    if len(cache._attends) >= 256:
        cache._attends.clear()
    cache._attends[key] = (p, info)
    return p, info


def decode_attention(q, cache: KVCache, page_table, lengths, scale: Optional[float] = None,
                     max_length: Optional[int] = None, out=None, lse=False, workspace=None, stream=None,
                     route: str = "auto"):
    """Attention of one new token per stream over its cached tokens.

    q [batch, heads, head_dim]; page_table int32 [batch, pages]; lengths int32
    [batch], the tokens each stream sees (the new one among them, once written);
    heads / kv_heads query heads share a kv head. scale is 1 / sqrt(head_dim)
    by default. max_length bounds the lengths (default: what the table can
    hold); a close bound saves launching blocks for parts no stream reaches.
    A given workspace is contiguous, with at least attend_plan's workspace_bytes.
    Returns out [batch, heads, head_dim]; with lse (True, or a float32 tensor
    [batch, heads] to fill) the pair (out, lse), lse the logarithm of the sum
    of exponentials. A stream that sees nothing gets zeros and -infinity."""
    _check(q, "q", None, None, cache.device)
    _check(page_table, "page_table", None, torch.int32, cache.device)
    if out is not None:
        _check(out, "out", q.shape, q.dtype, cache.device)
    p, info = attend_plan(cache, q, page_table, scale, max_length, out, route)
    batch, heads = q.shape[0], q.shape[1]
    _check(lengths, "lengths", (batch,), torch.int32, cache.device)
    if batch > 1 and lengths.stride(0) != 1:
        raise ValueError("lengths must be contiguous")
    sh, ext = _launch_stream(stream, cache.device)
    owned = []
    if out is None:
        out = _empty(q.shape, q.dtype, cache.device)
        owned.append(out)
    lse_t = None
    if lse is True:
        lse_t = _empty((batch, heads), torch.float32, cache.device)
        owned.append(lse_t)
    elif lse is not False and lse is not None:
        _check(lse, "lse", (batch, heads), torch.float32, cache.device)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        lse_t = lse
    if workspace is None:
        if info.workspace_bytes:
            workspace = _empty((info.workspace_bytes,), torch.uint8, cache.device)
            owned.append(workspace)
    else:
        _check_workspace(workspace, info.workspace_bytes, cache.device)
    st = _on_device(cache.device, (_ready or lib()).convt_attend, ctypes.byref(p), q.data_ptr(), cache.k.data_ptr(),
                    cache.v.data_ptr(), _ptr(cache.k_scale), _ptr(cache.v_scale), page_table.data_ptr(), lengths.data_ptr(),
                    out.data_ptr(), _ptr(lse_t), _ptr(workspace), sh)
    if st:
        _raise(st, "convt_attend")
    if ext is not None:
        _tie_to_stream(owned, ext)
    return out if lse_t is None else (out, lse_t)


def q4_quantise(weight, group: int = 128) -> Tuple[torch.Tensor, torch.Tensor]:
    """4-bit weights of weight [n, k] for q4_matvec: (w, scales) with w uint8 [n, k / 2] and
    scales [n, k / group] of weight's type, each group's largest magnitude at 7
    steps. Done once, where weights are loaded (plain torch, any device)."""
    n, k = weight.shape
    if group < 8 or group % 8 or k % group:
        raise ValueError("group must be a multiple of 8 that divides k")
    g = weight.float().reshape(n, k // group, group)
    scales = (g.abs().amax(-1) / 7).to(weight.dtype)
    step = scales.float().unsqueeze(-1)
    codes = torch.where(step > 0, g / torch.where(step > 0, step, 1.0), 0.0)
    codes = (codes.round().clamp(-8, 7) + 8).to(torch.uint8).reshape(n, k // 2, 2)
    return codes[:, :, 0] | codes[:, :, 1] << 4, scales


def q4_matvec(x, w, scales, x_scale=None, y=None, stream=None, route: str = "auto"):
    """y[..., n] = x W^T for a few rows of x[..., k] and the 4-bit weights (w, scales) of
    q4_quantise: w uint8 [n, k / 2], the even k in the low bits, codes 0 .. 15 for -8 .. 7;
    scales [n, k / group]. x is of scales' type, or e4m3 codes with x_scale (float32,
    one per row), as rms_norm gives them. Returns y of scales' type."""
    _check(x, "x")
    device, dtype = x.device, scales.dtype
    code = _code(scales, "scales")
    _check(scales, "scales", None, None, device)
    if w.dim() != 2 or scales.dim() != 2:
        raise ValueError("w and scales must have two axes")
    n, half = w.shape
    k = 2 * half
    _check(w, "w", None, torch.uint8, device)
    groups = scales.shape[1]
    if scales.shape[0] != n or (k % groups if groups else k):
        raise ValueError(f"scales has shape {tuple(scales.shape)}, expected ({n}, k / group) for k = {k}")
    if not (w.is_contiguous() and scales.is_contiguous()):
        raise ValueError("w and scales must be contiguous")
    rows, xs = _rows(x, "x")
    if x.shape[-1] != k:
        raise ValueError(f"x has {x.shape[-1]} columns, expected {k}")
    quantised = x_scale is not None
    if x.dtype != (_E4M3 if quantised else dtype):
        raise ValueError(f"x must be {_E4M3 if quantised else dtype}")
    if quantised:
        _check(x_scale, "x_scale", x.shape[:-1], torch.float32, device)
        if not x_scale.is_contiguous():
            raise ValueError("x_scale must be contiguous")
    sh, ext = _launch_stream(stream, device)
    owned = []
    shape = x.shape[:-1] + (n,)
    if y is None:
        y = _empty(shape, dtype, device)
        owned.append(y)
        ys = n
    else:
        _check(y, "y", shape, dtype, device)
        ys = _rows(y, "y")[1]
    p = Q4Problem(rows, n, k, k // groups if groups else 8, xs, ys, code, 1 if quantised else 0, Q4_ROUTES[route], 0)
    st = _on_device(device, (_ready or lib()).convt_q4_matvec, ctypes.byref(p), x.data_ptr(), _ptr(x_scale), w.data_ptr(),
                    scales.data_ptr(), y.data_ptr(), sh)
    if st:
        _raise(st, "convt_q4_matvec")
    if ext is not None:
        _tie_to_stream(owned, ext)
    return y
