"""sv_paged_attention on the GPU against the oracle.

Tolerances.  With u = 2^-24 (binary32) and h = 2^-8 (bf16): a score is a sum of
head_dim exact products in binary32, off by at most (head_dim + 4) u size, size
the largest scale * sum |q_d k_d| of a row (the oracle returns it); an
exponential adds 2^-22.  So every weight is off by a factor within 1 +- e,
e = (head_dim + 4) u size + 2^-21, its rounding to bf16 for the product with the
values by h more, and a weighted mean by at most 2 e + 2 h of its spread
sum w |v| / sum w (h for the rounded weights, and the sums' own roundings, at
most one per block of 16 tokens, are far below the second h); the result is
rounded by h of itself.  The logarithm is off by e and 2^-21 of itself."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import attn as oa
from test_gpu_kv import I32, new_cache, tables, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


def fill(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for n in ("k", "v"):
        x = torch.randn(c[n + "_cache"].shape, generator=g, device="cuda")
        if c[n + "_scale"] is None:
            c[n + "_cache"].copy_(x.bfloat16())
        else:
            c[n + "_cache"].copy_((x * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
            c[n + "_scale"].copy_(torch.randint(118, 123, c[n + "_scale"].shape, generator=g, device="cuda"))
    return c


def call(q, c, table, start, total, **kw):
    return sv.sv_paged_attention(q, c["k_cache"], c["v_cache"], I32(table), I32(start), I32(total),
                                 k_scale=c["k_scale"], v_scale=c["v_scale"], want_lse=True, **kw)


def check(o, q, c, table, start, total, scale, window=0, rows=None):
    n = lambda x: x.double().cpu().numpy()
    w = oa.attention(n(q), dict(k=values(c, "k"), v=values(c, "v"), table=np.asarray(table)), start, total, scale, window)
    rows = np.arange(start[0], start[-1]) if rows is None else rows
    out, lse = n(o["out"])[rows], n(o["lse"])[rows]
    want, wl, spread, size = (w[k][rows] for k in ("out", "lse", "spread", "size"))
    e = (q.shape[2] + 4) * 2.0 ** -24 * size + 2.0 ** -21
    tol = (2 * e[..., None] + 2 * 2.0 ** -8) * spread + np.abs(want) * 2.0 ** -8
    assert np.isfinite(out).all()
    worst = (np.abs(out - want) - tol).max()
    assert worst <= 0, worst
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(lse), empty) and (out[empty] == 0).all()
    assert (np.abs(lse - wl)[~empty] <= (e + np.abs(wl) * 2.0 ** -21)[~empty]).all()
    return w


SHAPES = [  # new, lengths, page, kv heads, q heads, D
    ([1], [1], 16, 1, 1, 64),
    ([1], [700], 16, 2, 8, 128),
    ([1, 1, 1], [5, 64, 333], 64, 8, 32, 128),
    ([5, 5, 5, 5], [5, 200, 17, 129], 16, 2, 8, 128),
    ([17, 1, 9], [40, 300, 9], 32, 1, 8, 128),
    ([3, 0, 2], [260, 77, 2], 8, 4, 28, 64),
    ([2, 5], [33, 70], 1, 5, 5, 80),
    ([4, 1], [100, 31], 128, 2, 14, 96),
    ([7, 1], [90, 257], 32, 1, 2, 256),
    ([100], [100], 16, 2, 4, 64),
    ([65, 130, 1], [65, 200, 5], 64, 1, 4, 128),
    ([70, 3], [300, 3], 16, 2, 6, 256),
    ([33, 40], [80, 40], 32, 3, 3, 16),
    ([50], [60], 16, 1, 16, 112),
    ([300], [420], 64, 1, 1, 128),
]


@pytest.mark.parametrize("cache,order", [("bf16", "tokens"), ("e4m3", "heads")])
@pytest.mark.parametrize("hints", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention_matches_the_oracle(cache, order, hints, shape):
    new, total, page, heads, q_heads, D = SHAPES[shape]
    pages, table, start = tables(new, total, page, seed=shape)
    c = fill(new_cache(cache, pages, page, heads, D, order), shape)
    start = start + 2
    T = int(start[-1]) + 3
    g = torch.Generator(device="cuda").manual_seed(shape)
    q = torch.randn((T, q_heads, D), generator=g, device="cuda").bfloat16()
    out = dict(out=torch.full_like(q, 9.0), lse=torch.full((T, q_heads), 9.0, device="cuda"))
    kw = dict(max_q_len=max(new), max_kv_len=max(total)) if hints else {}
    o = call(q, c, table, start, total, out=out, **kw)
    check(o, q, c, table, start, total, D ** -0.5)
    for x in (o["out"], o["lse"]):  # rows of no request
        assert (x[:2] == 9.0).all() and (x[start[-1]:] == 9.0).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 200, 100000])
@pytest.mark.parametrize("new,total,heads,q_heads,D", [([1, 1, 5], [300, 2, 170], 2, 8, 128), ([150, 70], [150, 400], 1, 4, 64),
                                                       ([40], [400], 2, 2, 128)])
def test_attention_window(cache, window, new, total, heads, q_heads, D):
    pages, table, start = tables(new, total, 16, seed=window)
    c = fill(new_cache(cache, pages, 16, heads, D), window)
    q = torch.randn((start[-1], q_heads, D), device="cuda").bfloat16()
    for kw in ({}, dict(max_q_len=max(new), max_kv_len=max(total))):
        o = call(q, c, table, start, total, scale=0.2, window=window, **kw)
        check(o, q, c, table, start, total, 0.2, window)


@pytest.mark.parametrize("new", [3, 40, 150])
def test_attention_rows_that_see_nothing(new):
    """Lengths of zero and below the new rows' number, requests with absent pages alone, pages absent in between."""
    page = 16
    table = np.array([[0, 1, 2] + [8] * 13, [-1] * 16, [3, 99, 4] + [-7] * 13, [5] * 16, [6, 7] + [-1] * 14])
    total = [0, 40, 44, max(1, new - 2), 2 ** 31 - 1]
    start = np.arange(6) * new
    c = fill(new_cache("bf16", 9, page, 2, 128), new)
    q = torch.randn((5 * new, 4, 128), device="cuda").bfloat16()
    o = call(q, c, table, start, total)
    # the last request's length is beyond its table: its rows lie there too, and see what the table holds
    total[4] = 10 ** 6
    want = check(o, q, c, table, start, [0, 40, 44, total[3], 0], 128 ** -0.5, rows=np.arange(4 * new))
    assert np.isneginf(want["lse"][: 2 * new]).all()
    last = oa.attention(q.double().cpu().numpy()[4 * new:], dict(k=values(c, "k"), v=values(c, "v"), table=table[4:]),
                        [0, new], [10 ** 4], 128 ** -0.5)
    err = np.abs(o["out"][4 * new:].double().cpu().numpy() - last["out"])
    assert (err <= (2 * 2.0 ** -8 + 2.0 ** -14) * last["spread"] + np.abs(last["out"]) * 2.0 ** -8).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,q_heads,total", [(1, 4, 37), (5, 8, 37), (40, 4, 75), (150, 2, 150), (20, 1, 290)])
def test_attention_ignores_what_it_does_not_see(cache, new, q_heads, total):
    """NaN, infinities and extremes in slots behind the end, on other pages and in later new tokens change nothing."""
    page, D = 16, 128
    pages, table, start = tables([new], [total], page, spare=3)
    c = fill(new_cache(cache, pages, page, 1, D), 5)
    q = torch.randn((new, q_heads, D), device="cuda").bfloat16()
    clean = call(q, c, table, start, [total])
    check(clean, q, c, table, start, [total], D ** -0.5)
    half = total - new // 2  # places from here on are not seen by the first rows
    poison = {k: (None if v is None else v.clone()) for k, v in c.items()}
    for n in ("k", "v"):
        x = poison[n + "_cache"]
        bad = [float("nan"), float("inf"), float("-inf"), 3e38] if cache == "bf16" else [float("nan")]
        seen = {(int(table[0, j // page]), j % page) for j in range(half)}
        i = 0
        for p in range(pages):
            for s in range(page):
                if (p, s) not in seen:
                    x[p, s] = torch.full((1, D), bad[i % len(bad)], device="cuda").to(x.dtype)
                    if poison[n + "_scale"] is not None:
                        poison[n + "_scale"][p, :, s] = [255, 120, 254][i % 3]
                    i += 1
    o = call(q, poison, table, start, [total])
    rows = half - (total - new)  # rows at places below `half`
    assert torch.equal(o["out"][:rows], clean["out"][:rows]) and torch.equal(o["lse"][:rows], clean["lse"][:rows])
    if rows < new:
        assert not torch.isfinite(o["out"][rows:].float()).any()


@pytest.mark.parametrize("new", [1, 6, 130])
def test_attention_large_scores(new):
    """Scores up to thousands, and equal ones: the running maximum keeps every exponential in range."""
    pages, table, start = tables([new], [400], 32)
    c = fill(new_cache("bf16", pages, 32, 2, 64), 3)
    q = (torch.randn((new, 4, 64), device="cuda") * 100).bfloat16()
    q[0] = 0
    o = call(q, c, table, start, [400], scale=2.0)
    check(o, q, c, table, start, [400], 2.0)


def test_attention_strides():
    """Queries out of a fused projection, outputs into a wider buffer, head-major rows, a shared page table row."""
    new, total, D = [5, 40], [60, 64], 64
    pages, table, start = tables(new, total, 16)
    c = fill(new_cache("bf16", pages, 16, 2, D), 1)
    fused = torch.randn((45, 12, D), device="cuda").bfloat16()
    q = fused[:, 2:10]
    want = call(q.contiguous(), c, table, start, total)
    check(want, q, c, table, start, total, D ** -0.5)
    wide = torch.full((45, 20, D), 5.0, device="cuda").bfloat16()
    o = call(q, c, table, start, total, out=dict(out=wide[:, 8:16]))
    assert torch.equal(o["out"], want["out"]) and (wide[:, :8] == 5).all() and (wide[:, 16:] == 5).all()
    major = q.transpose(0, 1).contiguous().transpose(0, 1)
    om = torch.empty((8, 45, D), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    assert torch.equal(call(major, c, table, start, total, out=dict(out=om))["out"], want["out"])
    shared = I32(table[:1]).expand(2, -1)
    k = (c["k_cache"], c["v_cache"])
    a = sv.sv_paged_attention(q, *k, shared, I32(start), I32([60, 64]))
    b = sv.sv_paged_attention(q, *k, shared.contiguous(), I32(start), I32([60, 64]))
    assert torch.equal(a["out"], b["out"])


def test_attention_far_in_a_large_cache():
    """Pages whose elements lie beyond 2^32, in the cache's bytes and in its elements."""
    page, heads, D = 64, 8, 128
    pages = (1 << 32) // (page * heads * D) + 70
    c = {}
    for n in ("k", "v"):
        c[n + "_cache"] = torch.empty((pages, page, heads, D), device="cuda", dtype=torch.bfloat16)
        c[n + "_scale"] = None
    table = np.array([[pages - 1, 0, pages - 2, pages // 2 + 1], [pages - 3, 1, 2, pages - 4]])
    used = sorted({int(p) for p in table.flat})
    small = {n: torch.randn((len(used), page, heads, D), device="cuda").bfloat16() for n in ("k", "v")}
    for n in small:
        c[n + "_cache"][used] = small[n]
    near = np.array([[used.index(int(p)) for p in row] for row in table])
    s = dict(k_cache=small["k"], v_cache=small["v"], k_scale=None, v_scale=None)
    for new in (4, 90):
        q = torch.randn((2 * new, 16, D), device="cuda").bfloat16()
        x = torch.randn((2 * new, heads, D), device="cuda").bfloat16()
        start, total = [0, new, 2 * new], [250, 190]
        for cc, tt in ((c, table), (s, near)):
            sv.sv_kv_append(x, x * 2, cc["k_cache"], cc["v_cache"], I32(tt), I32(start), I32(total))
        far, close = call(q, c, table, start, total), call(q, s, near, start, total)
        assert torch.equal(far["out"], close["out"]) and torch.equal(far["lse"], close["lse"])
        rows = lambda cc, tt: sv.sv_kv_gather(cc["k_cache"], cc["v_cache"], I32(tt), I32([0, 250, 440]), 440)
        a, b = rows(c, table), rows(s, near)
        assert torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"])


def test_attention_is_deterministic_and_hints_change_roundings_only():
    new, total = [1, 5, 9, 1], [3000, 1700, 40, 9]
    pages, table, start = tables(new, total, 16)
    c = fill(new_cache("bf16", pages, 16, 2, 128), 8)
    q = torch.randn((16, 16, 128), device="cuda").bfloat16()
    first = call(q, c, table, start, total)
    for kw in ({}, dict(max_q_len=1), dict(max_q_len=9, max_kv_len=3000), dict(max_q_len=4000), dict(max_kv_len=10)):
        o, again = call(q, c, table, start, total, **kw), call(q, c, table, start, total, **kw)
        assert torch.equal(o["out"], again["out"]) and torch.equal(o["lse"], again["lse"])
        check(o, q, c, table, start, total, 128 ** -0.5)
        assert not kw or torch.allclose(o["out"].float(), first["out"].float(), rtol=0.05, atol=0.02)


def test_attention_of_many_short_requests():
    B = 700
    g = np.random.default_rng(5)
    new = g.integers(0, 4, B)
    total = new + g.integers(0, 60, B)
    pages, table, start = tables(new, total, 8)
    c = fill(new_cache("e4m3", pages, 8, 1, 64), 2)
    q = torch.randn((start[-1], 4, 64), device="cuda").bfloat16()
    o = call(q, c, table, start, total, max_q_len=3, max_kv_len=int(total.max()))
    check(o, q, c, table, start, total, 0.125)


def test_attention_empty_and_refusals():
    pages, table, start = tables([4], [30], 16)
    c = fill(new_cache("bf16", pages, 16, 2, 64), 1)
    q = torch.randn((4, 8, 64), device="cuda").bfloat16()
    a = (q, c["k_cache"], c["v_cache"], I32(table), I32(start), I32([30]))
    assert set(sv.sv_paged_attention(*a)) == {"out"}
    assert call(q[:0], c, table, [0, 0], [30])["out"].shape == (0, 8, 64)

    def swap(i, y):
        b = list(a)
        b[i] = y
        return b

    for i, y, err in ((0, q.float(), TypeError), (0, q[..., :32], ValueError), (0, q[0], ValueError), (5, I32([30, 1]), ValueError),
                      (4, I32([0, 4, 5]), ValueError), (1, c["k_cache"].float(), TypeError), (0, q.transpose(1, 2), ValueError),
                      (3, I32(table).long(), TypeError), (0, q.cpu(), ValueError)):
        with pytest.raises(err):
            sv.sv_paged_attention(*swap(i, y))
    for kw in (dict(scale=-1.0), dict(scale=float("nan")), dict(window=-1), dict(max_q_len=-1)):
        with pytest.raises(RuntimeError, match="invalid argument"):
            sv.sv_paged_attention(*a, **kw)
    with pytest.raises(RuntimeError, match="invalid argument"):
        sv.sv_paged_attention(*swap(0, q[:, :7]))  # 7 heads over 2
    with pytest.raises(RuntimeError, match="invalid argument"):
        flat = torch.randn(4 * 8 * 64 + 4, device="cuda").bfloat16()
        sv.sv_paged_attention(*swap(0, flat[4:].view(4, 8, 64)))  # 8-byte aligned
    with pytest.raises(ValueError):
        sv.sv_paged_attention(*a, out=dict(out=q[:3]))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 1024])
@pytest.mark.parametrize("new,total,heads,q_heads,D", [
    ([1, 3], [70, 200], 2, 8, 128), ([10, 2], [150, 44], 1, 4, 64), ([13], [90], 2, 6, 128), ([30], [77], 1, 1, 256),
    ([70, 5], [90, 170], 1, 2, 128), ([140], [150], 2, 2, 64), ([40], [140], 1, 4, 256),
])
def test_attention_page_sizes(cache, page, new, total, heads, q_heads, D):
    """Every kernel (16, 32, 64 and 128 rows) with pages from one token to more than the context."""
    pages, table, start = tables(new, total, page, seed=page)
    c = fill(new_cache(cache, pages, page, heads, D), page)
    q = torch.randn((start[-1], q_heads, D), device="cuda").bfloat16()
    o = call(q, c, table, start, total, max_q_len=max(new), max_kv_len=max(total))
    check(o, q, c, table, start, total, D ** -0.5)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,total,window,q_heads", [
    ([3], [3000], 0, 4), ([3], [3000], 700, 4), ([9, 1], [2600, 30], 0, 8), ([20], [2900], 1000, 4),
    ([60, 2], [2100, 1800], 0, 4), ([50], [4000], 300, 4), ([1, 1, 1], [5000, 700, 0], 0, 2),
])
def test_attention_long_contexts_in_splits(cache, new, total, window, q_heads):
    """Contexts that are divided, windows that begin in a later split, requests that need none of the splits."""
    pages, table, start = tables(new, total, 32, seed=len(new))
    c = fill(new_cache(cache, pages, 32, 1, 128), 7)
    q = torch.randn((start[-1], q_heads, 128), device="cuda").bfloat16()
    size = sv.sv_paged_attention_workspace_size(len(new), int(start[-1]), q_heads, 1, 128, max(new), max(total))
    assert size > 256
    o = call(q, c, table, start, total, window=window, max_q_len=max(new), max_kv_len=max(total))
    check(o, q, c, table, start, total, 128 ** -0.5, window)


@pytest.mark.parametrize("q_heads", [2, 16])
def test_attention_of_one_long_request_among_short_ones(q_heads):
    """A request with far more rows than the average (and than a wrong hint says): its workgroups go on to its other
    tiles."""
    new, total = [1, 300, 1, 0, 2, 1, 1, 1], [40, 310, 1, 9, 77, 500, 3, 64]
    pages, table, start = tables(new, total, 16)
    c = fill(new_cache("bf16", pages, 16, 2, 64), 1)
    q = torch.randn((start[-1], q_heads, 64), device="cuda").bfloat16()
    for kw in ({}, dict(max_q_len=1), dict(max_q_len=300), dict(max_kv_len=3)):
        o = call(q, c, table, start, total, **kw)
        check(o, q, c, table, start, total, 0.125)


def test_attention_of_keys_and_values_in_one_tensor():
    """Keys and values interleaved in one allocation, and a cache with more heads' room than it has."""
    new, total, page, D = [3, 40], [60, 64], 16, 128
    pages, table, start = tables(new, total, page)
    for view in (lambda t: (t[:, 0], t[:, 1]), lambda t: (t[:, 0, :, 1:3], t[:, 1, :, :2])):
        both = torch.randn((pages, 2, page, 4, D), device="cuda").bfloat16()
        k, v = view(both)
        heads = k.shape[2]
        c = dict(k_cache=k, v_cache=v, k_scale=None, v_scale=None)
        x = torch.randn((43, heads, D), device="cuda").bfloat16()
        sv.sv_kv_append(x, -x, k, v, I32(table), I32(start), I32(total))
        q = torch.randn((43, 2 * heads, D), device="cuda").bfloat16()
        o = call(q, c, table, start, total)
        check(o, q, c, table, start, total, D ** -0.5)
        back = sv.sv_kv_gather(k, v, I32(table), I32(start), 43, kv_begin=I32([57, 24]))
        assert torch.equal(back["k"], x) and torch.equal(back["v"], -x)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_of_many_heads(new):
    """1024 query heads over 512 and over one key head."""
    for heads in (512, 1):
        pages, table, start = tables([new], [60], 16)
        c = fill(new_cache("bf16", pages, 16, heads, 16), 1)
        q = torch.randn((new, 1024, 16), device="cuda").bfloat16()
        o = call(q, c, table, start, [60])
        check(o, q, c, table, start, [60], 0.25)


@pytest.mark.parametrize("new,q_heads", [(1, 4), (12, 4), (140, 2)])
def test_attention_of_queries_that_are_not_finite(new, q_heads):
    """A row's queries reach that row alone."""
    pages, table, start = tables([new], [200], 16)
    c = fill(new_cache("bf16", pages, 16, 1, 128), 1)
    q = torch.randn((new, q_heads, 128), device="cuda").bfloat16()
    clean = call(q, c, table, start, [200])
    q[new // 2, 1, 5] = float("nan")
    o = call(q, c, table, start, [200])
    hit = torch.zeros((new, q_heads), dtype=torch.bool, device="cuda")
    hit[new // 2, 1] = True
    assert torch.isnan(o["out"][hit]).all() and torch.isnan(o["lse"][hit]).all()
    assert torch.equal(o["out"][~hit], clean["out"][~hit]) and torch.equal(o["lse"][~hit], clean["lse"][~hit])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,q_heads,total", [(4, 4, 900), (8, 4, 300), (8, 4, 320), (160, 2, 704), (320, 1, 1344)])
@pytest.mark.parametrize("seed", range(3))
def test_attention_of_a_row_keeps_its_bits_when_a_later_token_changes(cache, new, q_heads, total, seed):
    """Also where the later rows of its tile see a score far above all others."""
    pages, table, start = tables([new], [total], 16, seed=new)
    c = fill(new_cache(cache, pages, 16, 1, 128), new + seed)
    g = torch.Generator(device="cuda").manual_seed(new + seed)
    q = torch.randn((new, q_heads, 128), generator=g, device="cuda").bfloat16()
    kw = dict(max_q_len=new, max_kv_len=total, scale=0.05)
    a = call(q, c, table, start, [total], **kw)
    page, slot = int(table[0][(total - 1) // 16]), (total - 1) % 16
    key = c["k_cache"][page, slot, 0]
    key.copy_((q[-1, 0].float() * 100).to(key.dtype))
    b = call(q, c, table, start, [total], **kw)
    for n in ("out", "lse"):
        assert torch.equal(a[n][:-1], b[n][:-1]), n
        assert not torch.equal(a[n][-1], b[n][-1]), n
    check(b, q, c, table, start, [total], 0.05)


def test_attention_strides_of_dimensions_of_one():
    pages, table, start = tables([1], [70], 16, seed=1)
    c = fill(new_cache("bf16", pages, 16, 1, 64), 1)
    q = torch.randn((1, 4, 64), device="cuda").bfloat16()
    odd = lambda x: torch.as_strided(x, x.shape, (777, x.stride(1), 1))
    out = dict(out=odd(torch.zeros_like(q)))
    o = call(odd(q), c, table, start, [70], out=out)
    check(o, q, c, table, start, [70], 0.125)
    q1 = torch.randn((1, 1, 64), device="cuda").bfloat16()
    o = call(torch.as_strided(q1, (1, 1, 64), (777, 5, 1)), c, table, start, [70])
    check(o, q1, c, table, start, [70], 0.125)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("batch,new,heads,q_heads,D,window", [(300, 5, 2, 16, 64, 0), (70, 1, 8, 128, 128, 0),
                                                             (260, 3, 4, 16, 256, 18000), (2200, 4, 4, 32, 16, 0)])
def test_attention_of_a_few_long_contexts_among_many_short_ones(cache, batch, new, heads, q_heads, D, window):
    """Few of the rows are split; requests without rows, of one, and with more than the hint says are among them."""
    rng = np.random.default_rng(batch)
    n = np.full(batch, new)
    n[rng.integers(0, batch, 20)] = 0
    n[rng.integers(0, batch, 10)] = 1
    n[batch // 2] = new + 2
    total = n + rng.integers(0, 40, batch)
    total[[1, batch // 3, batch // 2, batch - 1]] += [17000, 33000, 20000, 9000]
    pages, table, start = tables(n.tolist(), total.tolist(), 64, seed=batch)
    c = fill(new_cache(cache, pages, 64, heads, D), batch)
    g = torch.Generator(device="cuda").manual_seed(batch)
    q = torch.randn((start[-1], q_heads, D), generator=g, device="cuda").bfloat16()
    o = call(q, c, table, start, total, window=window, max_q_len=new, max_kv_len=int(total.max()))
    check(o, q, c, table, start, total, D ** -0.5, window)
