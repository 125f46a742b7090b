"""Oracle of normed heads and of a cache's pages - TEST INFRASTRUCTURE ONLY (see
package doc).

Plain float64 numpy and python lists, one step at a time, from the definitions:

* a head's row x becomes R(x r w), r = (mean x^2 + eps)^-1/2, R the rotation of
  ``oracle.attn.rope``; its gradients by the chain rule, matrix by matrix;
* a row at place p sees the tokens j <= p of its request, with a window those with
  j > p - window or j < sinks; the first tokens of a group's requests are those
  of its first request's row of the page table;
* pages of a cache move between requests' rows of a page table and a stack, one
  page at a time.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import attn as oa


def norm_rope(x, w, eps, positions, f, layout="half", mscale=1.0):
    """Rows float64 [T, heads, D] normed and turned."""
    x = np.asarray(x, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return oa.rope(x * r * w, positions, f, layout, mscale)


def norm_rope_backward(x, w, eps, dy, positions, f, layout="half", mscale=1.0):
    """(dx, dw) from dy: through the rotation, the weights, and the norm, whose derivative of component j by component i
    is r (i == j) - r^3 x_i x_j / D."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = oa.rope(dy, positions, f, layout, mscale, backward=True)
    dw = (g * x * r).sum((0, 1))
    g = g * w
    return r * g - r ** 3 * x * (g * x).sum(-1, keepdims=True) / D, dw


def pages(table, held, free, kv_len, page_size, capacity, shared=None):
    """Moves pages in place: ``table`` rows (lists) of max_pages entries, ``held`` list, ``free`` the stack (list).
    Returns ``granted``."""
    B = len(held)
    most = len(table[0]) if B else 0
    need, fits = [], []
    for b in range(B):
        held[b] = min(max(held[b], 0), most)
        n = -(-max(int(kv_len[b]), 0) // page_size)
        fits.append(n <= most)
        need.append(max(n, min(int(shared[b]), held[b])) if shared is not None else n)
    back = []
    for b in range(B):
        if not fits[b]:
            continue
        for i in range(need[b], held[b]):
            back.append(table[b][i])
            table[b][i] = -1
    free.extend(back[::-1])
    del free[capacity:]
    granted, spent, left = [], 0, len(free)
    for b in range(B):
        lack = max(need[b] - held[b], 0) if fits[b] else 0
        spent += lack
        ok = fits[b] and (lack == 0 or spent <= left)
        granted.append(int(ok))
        if ok:
            for i in range(held[b], need[b]):
                table[b][i] = free.pop()
            held[b] = need[b]
    return granted


def slots(table, held, kv_len, query_start, page_size, capacity):
    """(slots, positions) of each row of a request, as lists; the rows are query_start[0] .. query_start[B] - 1."""
    where, place = [], []
    for b in range(len(held)):
        n = query_start[b + 1] - query_start[b]
        for i in range(n):
            p = max(int(kv_len[b]), 0) - n + i
            place.append(p)
            page = table[b][p // page_size] if 0 <= p // page_size < held[b] else -1
            where.append(page * page_size + p % page_size if 0 <= page < capacity else -1)
    return where, place


def attention(q, cache, query_start, kv_len, scale, window=0, sinks=0, group_start=(0,), shared_len=()):
    """As ``oracle.attn.attention``, with sinks and with groups of requests that share their first tokens."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    g = Hq // cache["k"].shape[2]
    out, spread = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, size = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        first, shared = b, 0
        for i, n in enumerate(shared_len):
            if group_start[i] <= b < group_start[i + 1]:
                first, shared = group_start[i], n
        for r in range(query_start[b], query_start[b + 1]):
            p = oa.place_of(query_start, np.maximum(kv_len, 0), b, r - query_start[b])
            seen = [j for j in range(p + 1) if window == 0 or j > p - window or j < sinks]
            at = [oa.slot_of(cache, first if j < shared else b, j) for j in seen]
            at = [x for x in at if x is not None]
            if not at:
                out[r], spread[r], lse[r] = 0, 0, -np.inf
                continue
            k, v = (cache[n][[x[0] for x in at], [x[1] for x in at]] for n in "kv")
            for h in range(Hq):
                s = scale * (k[:, h // g] @ q[r, h])
                top = s.max()
                w = np.exp(s - top)
                lse[r, h] = top + math.log(w.sum())
                out[r, h] = (w @ v[:, h // g]) / w.sum()
                spread[r, h] = (w @ np.abs(v[:, h // g])) / w.sum()
                size[r, h] = scale * (np.abs(k[:, h // g]) @ np.abs(q[r, h])).max()
    return dict(out=out, lse=lse, spread=spread, size=size)
