"""Oracle of the rotary, cache and attention operators - TEST INFRASTRUCTURE
ONLY (see package doc).

Plain float64 numpy, one step at a time, from the formulas:

* pair i of the turned channels of a row at position p is multiplied, as a
  complex number, by mscale * exp(j p f_i);
* an 8-bit row stands for code * 2^e with e the least integer in -117..127 such
  that its largest finite magnitude is at most 448 * 2^e (e = -9 for a row of
  zeros), every code the nearest value of the type (1 sign, 4 exponent, 3
  mantissa bits, bias 7), ties to the even code; what is not finite is NaN;
* row i of a request's n new rows is at place kv_len - n + i, and sees the
  tokens j <= place (j > place - window if there is a window) that the cache
  holds: softmax of scale * q.k over them, weights times v.

A cache is a dict: ``k``, ``v`` float64 [pages, page_size, heads, D], the values
it stands for, ``table`` int [B, max_pages].
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rotary, base=10000.0, scaling="plain", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """(f [rotary / 2], mscale)."""
    pairs = rotary // 2
    if scaling == "base":
        base = base * factor ** (rotary / (rotary - 2))
    f = np.array([1.0 / base ** (2 * i / rotary) for i in range(pairs)])
    if scaling in ("plain", "base"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    slow = f / factor
    if scaling == "bands":  # share kept by the number of turns over the original length
        turns = original_len / (2 * math.pi / f)
        share = np.clip((turns - low) / (high - low), 0, 1)
        return (1 - share) * slow + share * f, 1.0
    # ramp: share given up by the pair index, from the pair that turns `high` times to the one that turns `low` times
    index = lambda n: rotary * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(base))
    a = max(math.floor(index(high)), 0)
    b = min(math.ceil(index(low)), rotary - 1)
    if b <= a:
        b = a + 0.001
    given = np.clip((np.arange(pairs) - a) / (b - a), 0, 1)
    return given * slow + (1 - given) * f, 0.1 * math.log(factor) + 1.0


def rope(x, positions, f, layout="half", mscale=1.0, backward=False):
    """x float64 [T, heads, D] with its first 2 len(f) channels turned."""
    x = np.asarray(x, np.float64)
    r = 2 * len(f)
    # the angle's whole turns are dropped in extended precision
    t = np.asarray(positions, np.longdouble)[:, None] * np.asarray(f, np.longdouble)[None]
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    t = (t - np.rint(t / two_pi) * two_pi).astype(np.float64)
    z = mscale * np.exp((-1j if backward else 1j) * t)[:, None, :]
    y = x.copy()
    if layout == "half":
        w = (x[..., : r // 2] + 1j * x[..., r // 2: r]) * z
        y[..., : r // 2], y[..., r // 2: r] = w.real, w.imag
    else:
        w = (x[..., 0:r:2] + 1j * x[..., 1:r:2]) * z
        y[..., 0:r:2], y[..., 1:r:2] = w.real, w.imag
    return y


def e4m3_values():
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c >> 7 else 1.0, (c >> 3) & 15, c & 7
        out[c] = s * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        if e == 15 and m == 7:
            out[c] = np.nan
    return out


def quantise(rows):
    """(codes uint8 [..., D], e int [...]) of rows float64 [..., D]."""
    rows = np.asarray(rows, np.float64)
    values = e4m3_values()[:127]  # ascending, 0 .. 448
    top = np.where(np.isfinite(rows), np.abs(rows), 0).max(-1)
    e = np.empty(top.shape, int)
    for i in np.ndindex(top.shape):
        if top[i] == 0:
            e[i] = -9
            continue
        n = -117
        while top[i] > 448 * 2.0 ** n:
            n += 1
        e[i] = n
    x = rows / 2.0 ** e[..., None]
    a = np.where(np.isfinite(x), np.abs(x), 0)
    above = np.clip(np.searchsorted(values, a), 1, 126)
    down, up = a - values[above - 1], values[above] - a
    code = np.where((up < down) | ((up == down) & (above % 2 == 0)), above, above - 1)
    code = np.where(np.isfinite(rows), code, 127)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8), e


def place_of(query_start, kv_len, b, i):
    return int(kv_len[b]) - (int(query_start[b + 1]) - int(query_start[b])) + i


def slot_of(cache, b, place):
    """(page, slot) of a place, or None where the cache holds nothing."""
    size = cache["k"].shape[1]
    table = cache["table"]
    if place < 0 or place // size >= table.shape[1]:
        return None
    page = int(table[b, place // size])
    return (page, place % size) if 0 <= page < cache["k"].shape[0] else None


def gather(cache, row_start, rows, kv_begin=None):
    """(k, v) float64 [rows, heads, D]; NaN in rows that are not written."""
    heads, D = cache["k"].shape[2:]
    out = {n: np.full((rows, heads, D), np.nan) for n in ("k", "v")}
    for b in range(len(row_start) - 1):
        for r in range(row_start[b], row_start[b + 1]):
            at = slot_of(cache, b, (0 if kv_begin is None else int(kv_begin[b])) + r - row_start[b])
            for n in out:
                out[n][r] = 0 if at is None else cache[n][at]
    return out


def attention(q, cache, query_start, kv_len, scale, window=0):
    """out float64 [T, Hq, D], lse [T, Hq], and for error bounds: spread = sum w |v| / sum w [T, Hq, D] and size, the
    largest scale * sum |q_d k_d| of a seen token [T, Hq].  NaN in rows of no request."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    g = Hq // cache["k"].shape[2]
    out, spread = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, size = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        held = [(j, slot_of(cache, b, j)) for j in range(max(0, int(kv_len[b])))]
        held = [(j, at) for j, at in held if at is not None]
        j = np.array([h[0] for h in held], int)
        pages = np.array([h[1][0] for h in held], int)
        slots = np.array([h[1][1] for h in held], int)
        for r in range(query_start[b], query_start[b + 1]):
            p = place_of(query_start, kv_len, b, r - query_start[b])
            see = j <= p
            if window > 0:
                see &= j > p - window
            if not see.any():
                out[r], spread[r], lse[r] = 0, 0, -np.inf
                continue
            k, v = cache["k"][pages[see], slots[see]], cache["v"][pages[see], slots[see]]
            for h in range(Hq):
                s = scale * (k[:, h // g] @ q[r, h])
                top = s.max()
                w = np.exp(s - top)
                lse[r, h] = top + math.log(w.sum())
                out[r, h] = (w @ v[:, h // g]) / w.sum()
                spread[r, h] = (w @ np.abs(v[:, h // g])) / w.sum()
                size[r, h] = scale * (np.abs(k[:, h // g]) @ np.abs(q[r, h])).max()
    return dict(out=out, lse=lse, spread=spread, size=size)
