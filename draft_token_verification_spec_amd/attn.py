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
import functools
import struct
from typing import Optional

import torch

from . import SV_BF16, SV_F32, _check, _load

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
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (missing where torch has no device support)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


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
#
# A call's own time on the host is that of a few microseconds' kernel, so the
# checks read each attribute once and devices are compared by their index.

def _tensor(name: str, t) -> int:
    """The index of the HIP device that holds ``t``."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must live on a HIP device (got {t.device})")
    return dev


def _refuse(dev: int, name: str, t, dtype):
    """Why ``t`` is not a tensor of ``dtype`` on device ``dev``."""
    if _tensor(name, t) != dev:
        raise ValueError(f"{name} must live on the call's HIP device cuda:{dev} (got {t.device})")
    raise TypeError(f"{name} must be {dtype} (got {t.dtype})")


def _array(dev: int, name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple) -> int:
    """A contiguous array of exactly ``shape``; its address."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != dtype:
        _refuse(dev, name, t, dtype)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)} (got {list(t.shape)})")
    return t.data_ptr()


def _rows(dev: int, name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple):
    """Rows [T, heads, D] with contiguous channels; (address, row stride, head stride)."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != dtype:
        _refuse(dev, name, t, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    token, head, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have unit stride along the channels")
    return t.data_ptr(), token, head


def _three(name: str, t: torch.Tensor) -> tuple:
    """(T, heads, D) of rows."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [rows, heads, head_dim] (got {list(shape)})")
    if shape[0] > SV_ATTN_MAX_ROWS:
        raise ValueError(f"{name} has {shape[0]} rows, a call has at most {SV_ATTN_MAX_ROWS}")
    return shape


def _wide(n: int) -> int:
    """A window or hint as the C call's int, which would wrap around: what is beyond it says no more than its ends."""
    return n if -1 <= n <= 0x7FFFFFFF else 0x7FFFFFFF if n > 0 else -1


def _new(shape: tuple, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """A contiguous [T, heads, D] tensor (torch.empty takes a third longer)."""
    T, heads, D = shape
    return torch.empty_strided(shape, (heads * D, D, 1), dtype=dtype, device=device)


def _dtype_code(name: str, dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return SV_BF16
    if dtype == torch.float32:
        return SV_F32
    raise TypeError(f"{name} must be bfloat16 or float32 (got {dtype})")


def _layout(layout: str) -> int:
    try:
        return SV_ROPE_LAYOUTS[layout]
    except (KeyError, TypeError):
        raise ValueError(f"layout must be one of {sorted(SV_ROPE_LAYOUTS)} (got {layout!r})") from None


def _freq(dev: int, freq: Optional[torch.Tensor]):
    """(address, turned channels) of a frequency table."""
    if freq is None:
        return None, 0
    if not isinstance(freq, torch.Tensor) or freq.get_device() != dev or freq.dtype != torch.float64:
        _refuse(dev, "freq", freq, torch.float64)
    if freq.dim() != 1 or not freq.is_contiguous():
        raise ValueError("freq must be a contiguous 1-D table")
    return freq.data_ptr(), 2 * freq.shape[0]


# sv_paged_cache, as bytes: heads and head_dim are fields 1 and 2, max_pages and page_size 5 and 3
_CACHE = struct.Struct("@6iPqPP6qPP")


def _paged(dev: int, B: int, k_cache, v_cache, page_table, k_scale, v_scale):
    """(sv_paged_cache, heads, head_dim, page table's tokens)."""
    _tensor("k_cache", k_cache)
    kind = k_cache.dtype
    if kind != torch.bfloat16 and kind != torch.float8_e4m3fn or k_cache.get_device() != dev:
        _refuse(dev, "k_cache", k_cache, "bfloat16 or float8_e4m3fn")
    if not isinstance(v_cache, torch.Tensor) or v_cache.get_device() != dev or v_cache.dtype != kind:
        _refuse(dev, "v_cache", v_cache, kind)
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, heads, head_dim], both alike")
    pages, page_size, heads, D = shape
    kp, kt, kh, k1 = k_cache.stride()
    vp, vt, vh, v1 = v_cache.stride()
    if k1 != 1 or v1 != 1:
        raise ValueError("k_cache and v_cache must have unit stride along the channels")
    if not isinstance(page_table, torch.Tensor) or page_table.get_device() != dev or page_table.dtype != torch.int32:
        _refuse(dev, "page_table", page_table, torch.int32)
    tshape = page_table.shape
    if len(tshape) != 2 or tshape[0] != B:
        raise ValueError(f"page_table must be [{B}, max_pages] (got {list(tshape)})")
    max_pages = tshape[1]
    table_stride, one = page_table.stride()
    if one != 1 and max_pages > 1:
        raise ValueError("page_table must have unit stride along the pages")
    # strides along dimensions of one element say nothing: torch may give any
    if B <= 1:
        table_stride = max_pages
    if page_size == 1:
        kt = vt = D
    if heads == 1:
        kh = vh = D
    if pages <= 1:
        kp = vp = page_size * heads * D
    if kind == torch.float8_e4m3fn:
        if k_scale is None or v_scale is None:
            raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale")
        code = SV_E4M3
        ks = _array(dev, "k_scale", k_scale, torch.uint8, (pages, heads, page_size))
        vs = _array(dev, "v_scale", v_scale, torch.uint8, (pages, heads, page_size))
    else:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        code, ks, vs = SV_BF16, 0, 0
    return _CACHE.pack(code, heads, D, page_size, pages, max_pages, page_table.data_ptr(), table_stride,
                       k_cache.data_ptr(), v_cache.data_ptr(), kp, kt, kh, vp, vt, vh, ks, vs), heads, D, \
        max_pages * page_size


def _call(dev: int, what: str, *args):
    """Call the C entry point on the device's current stream, with the device current."""
    if _current_device() == dev:
        status = getattr(_lib or _attn_lib(), what)(_stream_of(dev), *args)
    else:
        with torch.cuda.device(dev):
            status = getattr(_lib or _attn_lib(), what)(_stream_of(dev), *args)
    if status != 0:
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
    dev = _tensor("x", x)
    shape = T, heads, D = _three("x", x)
    dtype = x.dtype
    code = _dtype_code("x", dtype)
    xr = _rows(dev, "x", x, dtype, shape)
    pos = _array(dev, "positions", positions, torch.int64, (T,))
    fp, rotary = _freq(dev, freq)
    if out is None:
        out = _new(shape, dtype, x.device)
        orows = out.data_ptr(), heads * D, D
    else:
        orows = _rows(dev, "out", out, dtype, shape)
    _call(dev, "sv_rope", T, heads, D, rotary, _layout(layout), 1 if backward else 0, code, *xr, pos, fp, mscale,
          *orows)
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
    dev = _tensor("k", k)
    shape = T, heads, D = _three("k", k)
    _tensor("kv_len", kv_len)
    B = kv_len.numel()
    cache, cache_heads, cache_dim, _ = _paged(dev, B, k_cache, v_cache, page_table, k_scale, v_scale)
    if heads != cache_heads or D != cache_dim:
        raise ValueError(f"k is {list(shape)}, the cache has {cache_heads} heads of {cache_dim} channels")
    dtype = k.dtype
    code = _dtype_code("k", dtype)
    kr = _rows(dev, "k", k, dtype, shape)
    vr = _rows(dev, "v", v, dtype, shape)
    fp, rotary = _freq(dev, freq)
    pos = None if positions is None else _array(dev, "positions", positions, torch.int64, (T,))
    qs = _array(dev, "query_start", query_start, torch.int32, (B + 1,))
    kl = _array(dev, "kv_len", kv_len, torch.int32, (B,))
    o = {} if out is None else out
    q_heads, qr, qo = 0, (None, 0, 0), (None, 0, 0)
    if q is not None:
        _tensor("q", q)
        q_heads = _three("q", q)[1]
        qr = _rows(dev, "q", q, dtype, (T, q_heads, D))
        if "q" in o:
            qo = _rows(dev, "out['q']", o["q"], dtype, (T, q_heads, D))
        else:
            o["q"] = _new((T, q_heads, D), dtype, q.device)
            qo = o["q"].data_ptr(), q_heads * D, D
    _call(dev, "sv_kv_append", B, T, q_heads, code, rotary, _layout(layout), fp, mscale, pos, *qr, *qo, *kr, *vr, qs,
          kl, cache)
    return o


def sv_kv_gather(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, row_start: torch.Tensor,
                 rows: int, *, kv_begin: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                 out: Optional[dict] = None) -> dict:
    """Read tokens of a paged cache back as ``k``, ``v`` [rows, heads,
    head_dim] of ``dtype`` (bfloat16 or float32); see ``sv_kv_gather``.
    ``row_start`` int32 [B + 1]; ``kv_begin`` int32 [B], default 0.  Rows
    outside ``row_start`` are not written."""
    dev = _tensor("k_cache", k_cache)
    _tensor("row_start", row_start)
    B = row_start.numel() - 1
    if B < 0:
        raise ValueError("row_start must have B + 1 entries")
    cache, heads, D, _ = _paged(dev, B, k_cache, v_cache, page_table, k_scale, v_scale)
    rs = _array(dev, "row_start", row_start, torch.int32, (B + 1,))
    kb = None if kv_begin is None else _array(dev, "kv_begin", kv_begin, torch.int32, (B,))
    code = _dtype_code("dtype", dtype)
    o = {} if out is None else out
    if rows > SV_ATTN_MAX_ROWS:
        raise ValueError(f"{rows} rows, a call has at most {SV_ATTN_MAX_ROWS}")
    shape = (rows, heads, D)
    ptr = []
    for name in ("k", "v"):
        if name in o:
            ptr.append(_array(dev, f"out['{name}']", o[name], dtype, shape))
        else:
            t = o[name] = _new(shape, dtype, k_cache.device)
            ptr.append(t.data_ptr())
    _call(dev, "sv_kv_gather", B, rows, code, cache, rs, kb, *ptr)
    return o


@functools.lru_cache(maxsize=4096)
def sv_paged_attention_workspace_size(B: int, T: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int = 0,
                                      max_kv_len: int = 0) -> int:
    return int(_attn_lib().sv_paged_attention_workspace_size(B, T, q_heads, kv_heads, head_dim, _wide(max_q_len),
                                                             _wide(max_kv_len)))


def sv_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                       query_start: torch.Tensor, kv_len: torch.Tensor, *, scale: Optional[float] = None,
                       window: int = 0, k_scale: Optional[torch.Tensor] = None,
                       v_scale: Optional[torch.Tensor] = None, max_q_len: int = 0, max_kv_len: int = 0,
                       want_lse: bool = False, workspace: Optional[torch.Tensor] = None,
                       out: Optional[dict] = None) -> dict:
    """Causal attention of the new tokens ``q`` [T, q_heads, head_dim]
    (bfloat16) over a paged cache that holds them already; see
    ``sv_paged_attention``.  ``scale`` defaults to head_dim**-0.5; ``window``
    0: every earlier token.  Returns ``out`` (as q) and, if asked for, ``lse``
    float32 [T, q_heads]; rows of no request are not written.

    ``max_q_len``, ``max_kv_len``: the most new tokens of a request and the
    longest context, where known.  They change times, not results: without the
    first a request of far more rows than the average is slow, without the second
    (default: the page table's width) contexts are divided for the longest one
    that the table could hold.

    Without a ``workspace`` the call takes one from torch's allocator for its
    own duration: calls on different streams, and captured graphs, then share
    nothing.  Else a contiguous uint8 tensor of at least
    ``sv_paged_attention_workspace_size`` bytes, used by one call at a time."""
    dev = _tensor("q", q)
    shape = T, q_heads, D = _three("q", q)
    _tensor("kv_len", kv_len)
    B = kv_len.numel()
    cache, heads, cache_dim, tokens = _paged(dev, B, k_cache, v_cache, page_table, k_scale, v_scale)
    if cache_dim != D:
        raise ValueError(f"q is {list(shape)}, the cache has heads of {cache_dim} channels")
    qr = _rows(dev, "q", q, torch.bfloat16, shape)
    qs = _array(dev, "query_start", query_start, torch.int32, (B + 1,))
    kl = _array(dev, "kv_len", kv_len, torch.int32, (B,))
    o = {} if out is None else out
    device = q.device
    if "out" in o:
        orows = _rows(dev, "out['out']", o["out"], torch.bfloat16, shape)
    else:
        t = o["out"] = _new(shape, torch.bfloat16, device)
        orows = t.data_ptr(), q_heads * D, D
    lse = None
    if "lse" in o:
        lse = _array(dev, "out['lse']", o["lse"], torch.float32, (T, q_heads))
    elif want_lse:
        t = o["lse"] = torch.empty_strided((T, q_heads), (q_heads, 1), dtype=torch.float32, device=device)
        lse = t.data_ptr()
    if max_kv_len == 0:
        max_kv_len = tokens
    nbytes = sv_paged_attention_workspace_size(B, T, q_heads, heads, D, max_q_len, max_kv_len)
    ws = None
    if workspace is None:
        if nbytes > 256:
            ws = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=device)
    else:
        ws = workspace
        _array(dev, "workspace", ws, torch.uint8, (ws.numel(),))
        nbytes = ws.numel()
    _call(dev, "sv_paged_attention", B, T, q_heads, *qr, cache, qs, kl, _wide(max_q_len), _wide(max_kv_len),
          D ** -0.5 if scale is None else scale, _wide(window), *orows, lse, None if ws is None else ws.data_ptr(), nbytes)
    return o
