"""Binding of ``include/specverify_attn.h``: rotary positions, a paged cache of
keys and values, and the attention of new tokens over it.

Argument marshalling only, as the rest of the package; the names are those of
the C entry points, and the package exports them.  A cache is a pair of tensors
``k_cache``, ``v_cache`` [num_pages, page_size, heads, head_dim] (any strides
with contiguous channels, so a [num_pages, heads, page_size, head_dim] cache is
passed as its ``transpose(1, 2)``): bfloat16, or float8_e4m3fn with ``k_scale``,
``v_scale`` uint8 [num_pages, heads, page_size].  ``page_table`` is int32
[B, max_pages], ``query_start`` int32 [B + 1], ``kv_len`` int32 [B].
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import SV_BF16, SV_F32, Workspace, _check, _load, _need

__all__ = [
    "SV_E4M3",
    "SV_ATTN_MAX_HEAD_DIM",
    "SV_ATTN_MAX_HEADS",
    "SV_ATTN_MAX_PAGE",
    "SV_ATTN_MAX_TOKENS",
    "SV_ATTN_MAX_ROWS",
    "SV_ROPE_LAYOUTS",
    "SV_ROPE_SCALINGS",
    "sv_rope_frequencies",
    "sv_rope",
    "sv_kv_append",
    "sv_kv_gather",
    "sv_paged_attention",
    "sv_paged_attention_workspace_size",
]

SV_E4M3 = 2
SV_ATTN_MAX_HEAD_DIM = 256
SV_ATTN_MAX_HEADS = 1024
SV_ATTN_MAX_PAGE = 65536
SV_ATTN_MAX_TOKENS = 1073741824
SV_ATTN_MAX_ROWS = 1 << 23
SV_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
SV_ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "ramp": 3, "bands": 4}

_p = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_f = ctypes.c_float
_d = ctypes.c_double


class _PagedCache(ctypes.Structure):  # sv_paged_cache
    _fields_ = [("dtype", _i), ("heads", _i), ("head_dim", _i), ("page_size", _i), ("num_pages", _i),
                ("max_pages", _i), ("page_table", _p), ("page_table_stride", _i64), ("k", _p), ("v", _p),
                ("k_page_stride", _i64), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_page_stride", _i64), ("v_token_stride", _i64), ("v_head_stride", _i64),
                ("k_scale", _p), ("v_scale", _p)]


_SIGNATURES = {
    "sv_rope_frequencies": (_i, [_i, _d, _i, _d, _d, _d, _d, _p, _p]),
    "sv_rope": (_i, [_p, _i, _i, _i, _i, _i, _i, _i, _p, _i64, _i64, _p, _p, _f, _p, _i64, _i64]),
    "sv_kv_append": (_i, [_p, _i, _i, _i, _i, _i, _i, _p, _f, _p, _p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p,
                          _i64, _i64, _p, _p, _p]),
    "sv_kv_gather": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _p]),
    "sv_paged_attention_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "sv_paged_attention": (_i, [_p, _i, _i, _i, _p, _i64, _i64, _p, _p, _p, _i, _i, _f, _i, _p, _i64, _i64, _p, _p,
                                _sz]),
}

_lib = None


def _attn_lib():
    global _lib
    if _lib is None:
        lib = _load()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _on(dev: torch.device, name: str, t: torch.Tensor, *dtypes):
    """``t`` is on the call's device, of one of ``dtypes``."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev or dev.type != "cuda":
        raise ValueError(f"{name} must live on the call's HIP device (got {t.device}, the call is on {dev})")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))} (got {t.dtype})")


def _array(dev: torch.device, name: str, t: torch.Tensor, dtype: torch.dtype, *shape) -> int:
    """A contiguous array of exactly ``shape``; its address."""
    _on(dev, name, t, dtype)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)} (got {list(t.shape)})")
    return t.data_ptr()


def _rows(dev: torch.device, name: str, t: torch.Tensor, dtype: torch.dtype, T: int, heads: int, D: int):
    """Rows [T, heads, D] with contiguous channels; (address, row stride, head stride)."""
    _on(dev, name, t, dtype)
    if t.shape != (T, heads, D):
        raise ValueError(f"{name} must be {[T, heads, D]} (got {list(t.shape)})")
    token, head, one = t.stride()
    if one != 1 and D > 1:
        raise ValueError(f"{name} must have unit stride along the channels")
    return t.data_ptr(), token, head


def _dtype_code(name: str, t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise TypeError(f"{name} must be bfloat16 or float32 (got {t.dtype})")


def _three(name: str, t: torch.Tensor):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, head_dim] (got {list(t.shape)})")
    return t.shape


def _layout(layout: str) -> int:
    try:
        return SV_ROPE_LAYOUTS[layout]
    except (KeyError, TypeError):
        raise ValueError(f"layout must be one of {sorted(SV_ROPE_LAYOUTS)} (got {layout!r})") from None


def _freq(dev: torch.device, freq: Optional[torch.Tensor]):
    """(address, turned channels) of a frequency table."""
    if freq is None:
        return None, 0
    _on(dev, "freq", freq, torch.float64)
    if freq.dim() != 1 or not freq.is_contiguous():
        raise ValueError("freq must be a contiguous 1-D table")
    return freq.data_ptr(), 2 * freq.shape[0]


def _paged(dev: torch.device, B: int, k_cache, v_cache, page_table, k_scale, v_scale) -> _PagedCache:
    _on(dev, "k_cache", k_cache, torch.bfloat16, torch.float8_e4m3fn)
    _on(dev, "v_cache", v_cache, k_cache.dtype)
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, heads, head_dim], both alike")
    pages, page_size, heads, D = k_cache.shape
    kp, kt, kh, k1 = k_cache.stride()
    vp, vt, vh, v1 = v_cache.stride()
    if k1 != 1 or v1 != 1:
        raise ValueError("k_cache and v_cache must have unit stride along the channels")
    _on(dev, "page_table", page_table, torch.int32)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be [{B}, max_pages] (got {list(page_table.shape)})")
    max_pages = page_table.shape[1]
    if page_table.stride(1) != 1 and max_pages > 1:
        raise ValueError("page_table must have unit stride along the pages")
    table_stride = page_table.stride(0) if B > 1 else max_pages
    fp8 = k_cache.dtype == torch.float8_e4m3fn
    if fp8:
        if k_scale is None or v_scale is None:
            raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale")
        ks = _array(dev, "k_scale", k_scale, torch.uint8, pages, heads, page_size)
        vs = _array(dev, "v_scale", v_scale, torch.uint8, pages, heads, page_size)
    else:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        ks = vs = None
    # strides along dimensions of one element say nothing: torch may give any
    if page_size == 1:
        kt, vt = D, D
    if heads == 1:
        kh, vh = D, D
    if pages <= 1:
        kp, vp = page_size * heads * D, page_size * heads * D
    return _PagedCache(SV_E4M3 if fp8 else SV_BF16, heads, D, page_size, pages, max_pages, page_table.data_ptr(),
                       table_stride, k_cache.data_ptr(), v_cache.data_ptr(), kp, kt, kh, vp, vt, vh, ks, vs)


def _call(dev: torch.device, what: str, *args):
    """Call the C entry point on the device's current stream, with the device current."""
    fn = getattr(_attn_lib(), what)
    stream = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev.index:
        status = fn(stream, *args)
    else:
        with torch.cuda.device(dev):
            status = fn(stream, *args)
    _check(status, what)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def sv_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "plain", *, factor: float = 1.0,
                        original_len: float = 0.0, low: float = 1.0, high: float = 32.0, device=None):
    """The frequency table of rotary positions, float64 [rotary_dim / 2] on
    ``device`` (default: the host), and the factor ``mscale`` of cos and sin;
    see ``sv_rope_frequencies``.  ``scaling``: "plain", "linear", "base",
    "ramp" or "bands"."""
    if scaling not in SV_ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(SV_ROPE_SCALINGS)} (got {scaling!r})")
    freq = torch.empty(max(0, rotary_dim // 2), dtype=torch.float64)
    mscale = ctypes.c_float()
    _check(_attn_lib().sv_rope_frequencies(int(rotary_dim), float(base), SV_ROPE_SCALINGS[scaling], float(factor),
                                           float(original_len), float(low), float(high), freq.data_ptr(),
                                           ctypes.addressof(mscale)), "sv_rope_frequencies")
    return (freq if device is None else freq.to(device)), mscale.value


def sv_rope(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, *, layout: str = "half",
            mscale: float = 1.0, backward: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotary positions on ``x`` [T, heads, head_dim] (bfloat16 or float32);
    see ``sv_rope``.  ``positions`` int64 [T]; ``freq`` float64 [turned
    channels / 2] on the device (``sv_rope_frequencies``).  ``backward``: ``x``
    is the gradient with respect to the output, and the gradient with respect
    to the input is returned.  ``out`` may be ``x``."""
    T, heads, D = _three("x", x)
    dev = x.device
    dtype = _dtype_code("x", x)
    xp, xt, xh = _rows(dev, "x", x, x.dtype, T, heads, D)
    pos = _array(dev, "positions", positions, torch.int64, T)
    fp, rotary = _freq(dev, freq)
    if out is None:
        out = torch.empty((T, heads, D), dtype=x.dtype, device=dev)
    op, ot, oh = _rows(dev, "out", out, x.dtype, T, heads, D)
    _call(dev, "sv_rope", T, heads, D, rotary, _layout(layout), int(bool(backward)), dtype, xp, xt, xh, pos, fp,
          mscale, op, ot, oh)
    return out


def sv_kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 page_table: torch.Tensor, query_start: torch.Tensor, kv_len: torch.Tensor, *,
                 q: Optional[torch.Tensor] = None, freq: Optional[torch.Tensor] = None, layout: str = "half",
                 mscale: float = 1.0, positions: Optional[torch.Tensor] = None,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 out: Optional[dict] = None) -> dict:
    """Append the new tokens' keys and values ``k``, ``v`` [T, heads, head_dim]
    (bfloat16 or float32) to a paged cache, in place, keys turned by their
    positions if ``freq`` is given; see ``sv_kv_append``.  ``q`` [T, q_heads,
    head_dim]: queries to turn likewise, returned as ``q`` (rows of no request
    are not written).  ``positions`` int64 [T], default: the tokens' places."""
    T, heads, D = _three("k", k)
    dev = k.device
    B = kv_len.numel()
    cache = _paged(dev, B, k_cache, v_cache, page_table, k_scale, v_scale)
    if (cache.heads, cache.head_dim) != (heads, D):
        raise ValueError(f"k is {list(k.shape)}, the cache has {cache.heads} heads of {cache.head_dim} channels")
    dtype = _dtype_code("k", k)
    kr = _rows(dev, "k", k, k.dtype, T, heads, D)
    vr = _rows(dev, "v", v, k.dtype, T, heads, D)
    fp, rotary = _freq(dev, freq)
    pos = None if positions is None else _array(dev, "positions", positions, torch.int64, T)
    qs = _array(dev, "query_start", query_start, torch.int32, B + 1)
    kl = _array(dev, "kv_len", kv_len, torch.int32, B)
    o = {} if out is None else out
    q_heads, qr, qo = 0, (None, 0, 0), (None, 0, 0)
    if q is not None:
        q_heads = _three("q", q)[1]
        qr = _rows(dev, "q", q, k.dtype, T, q_heads, D)
        _need(o, "q", (T, q_heads, D), q.dtype, dev)
        qo = _rows(dev, "out['q']", o["q"], k.dtype, T, q_heads, D)
    _call(dev, "sv_kv_append", B, T, q_heads, dtype, rotary, _layout(layout), fp, mscale, pos, *qr, *qo, *kr, *vr, qs,
          kl, ctypes.addressof(cache))
    return o


def sv_kv_gather(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, row_start: torch.Tensor,
                 rows: int, *, kv_begin: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                 out: Optional[dict] = None) -> dict:
    """Read tokens of a paged cache back as ``k``, ``v`` [rows, heads,
    head_dim] of ``dtype`` (bfloat16 or float32); see ``sv_kv_gather``.
    ``row_start`` int32 [B + 1]; ``kv_begin`` int32 [B], default 0.  Rows
    outside ``row_start`` are not written."""
    dev = k_cache.device
    if not isinstance(row_start, torch.Tensor) or row_start.numel() < 1:
        raise ValueError("row_start must be an int32 tensor of B + 1 entries")
    B = row_start.numel() - 1
    cache = _paged(dev, B, k_cache, v_cache, page_table, k_scale, v_scale)
    rs = _array(dev, "row_start", row_start, torch.int32, B + 1)
    kb = None if kv_begin is None else _array(dev, "kv_begin", kv_begin, torch.int32, B)
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be bfloat16 or float32 (got {dtype})")
    o = {} if out is None else out
    shape = (rows, cache.heads, cache.head_dim)
    _need(o, "k", shape, dtype, dev)
    _need(o, "v", shape, dtype, dev)
    ko = _array(dev, "out['k']", o["k"], dtype, *shape)
    vo = _array(dev, "out['v']", o["v"], dtype, *shape)
    _call(dev, "sv_kv_gather", B, rows, SV_BF16 if dtype == torch.bfloat16 else SV_F32, ctypes.addressof(cache), rs,
          kb, ko, vo)
    return o


def sv_paged_attention_workspace_size(B: int, T: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int = 0,
                                      max_kv_len: int = 0) -> int:
    return int(_attn_lib().sv_paged_attention_workspace_size(B, T, q_heads, kv_heads, head_dim, max_q_len,
                                                             max_kv_len))


def sv_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                       query_start: torch.Tensor, kv_len: torch.Tensor, *, scale: Optional[float] = None,
                       window: int = 0, k_scale: Optional[torch.Tensor] = None,
                       v_scale: Optional[torch.Tensor] = None, max_q_len: int = 0, max_kv_len: int = 0,
                       want_lse: bool = False, workspace: Optional[Workspace] = None,
                       out: Optional[dict] = None) -> dict:
    """Causal attention of the new tokens ``q`` [T, q_heads, head_dim]
    (bfloat16) over a paged cache that holds them already; see
    ``sv_paged_attention``.  ``scale`` defaults to head_dim**-0.5; ``window``
    0: every earlier token.  Returns ``out`` (as q) and, if asked for, ``lse``
    float32 [T, q_heads]; rows of no request are not written.

    Without a ``workspace`` the call takes one from torch's allocator for its
    own duration: calls on different streams, and captured graphs, then share
    nothing.  A Workspace serves one stream's calls, as everywhere."""
    T, q_heads, D = _three("q", q)
    dev = q.device
    B = kv_len.numel()
    cache = _paged(dev, B, k_cache, v_cache, page_table, k_scale, v_scale)
    if cache.head_dim != D:
        raise ValueError(f"q is {list(q.shape)}, the cache has heads of {cache.head_dim} channels")
    qp = _rows(dev, "q", q, torch.bfloat16, T, q_heads, D)
    qs = _array(dev, "query_start", query_start, torch.int32, B + 1)
    kl = _array(dev, "kv_len", kv_len, torch.int32, B)
    o = {} if out is None else out
    _need(o, "out", (T, q_heads, D), torch.bfloat16, dev)
    op = _rows(dev, "out['out']", o["out"], torch.bfloat16, T, q_heads, D)
    if want_lse:
        _need(o, "lse", (T, q_heads), torch.float32, dev)
    lp = _array(dev, "out['lse']", o["lse"], torch.float32, T, q_heads) if "lse" in o else None
    if max_kv_len == 0:
        max_kv_len = cache.max_pages * cache.page_size
    nbytes = _attn_lib().sv_paged_attention_workspace_size(B, T, q_heads, cache.heads, D, max_q_len, max_kv_len)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if workspace is None else workspace.get(dev, nbytes)
    _call(dev, "sv_paged_attention", B, T, q_heads, *qp, ctypes.addressof(cache), qs, kl, max_q_len, max_kv_len,
          D ** -0.5 if scale is None else scale, window, *op, lp, ws.data_ptr(), ws.numel())
    return o
