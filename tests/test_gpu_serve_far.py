"""The normed append and the attention with sinks and behind shared tokens over
caches whose pages or tokens lie beyond 32-bit offsets, over strided rows and
page tables, with hints of any kind, and over contexts of many tokens of which
few are seen: against the same call on a small cache, bit by bit."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import serve as osv
from test_gpu_attn import fill
from test_gpu_attn_sinks import N, within
from test_gpu_kv import I32, new_cache, tables, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


def calls(c, table, new, q, x, w, total, shared):
    """The three calls on one cache; their outputs and what the cache then holds."""
    B = len(total)
    start = I32([i * new for i in range(B + 1)])
    s = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    a = (c["k_cache"], c["v_cache"], I32(table))
    f, _ = sv.sv_rope_frequencies(q.shape[2], device="cuda")
    o = sv.sv_kv_append_normed(x, -x, *a, start, I32(total), q=q, freq=f, q_weight=w, k_weight=w, **s)
    sinks = sv.sv_paged_attention_sinks(o["q"], *a, start, I32(total), window=30, sinks=20, want_lse=True, **s)
    group = sv.sv_paged_attention_shared(o["q"], *a, start, I32(total), I32([0, B]), I32([shared]), want_lse=True, **s)
    rows = np.cumsum([0] + list(total))
    back = sv.sv_kv_gather(*a, I32(rows), int(rows[-1]), **s)
    return {**{"s_" + n: v for n, v in sinks.items()}, **{"g_" + n: v for n, v in group.items()}, **back, "q": o["q"]}


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("far", ["pages", "tokens", "more tokens"])
def test_far_apart(kind, far):
    """Pages behind 2^32 elements; 16 tokens just within, and just beyond, 2^32 bytes."""
    heads, D, size = 8, 128, 2 if kind == "bf16" else 1
    dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    word = torch.int16 if kind == "bf16" else torch.int8
    page = 64 if far == "pages" else 16
    if far == "pages":
        pages = (1 << 32) // (page * heads * D) + 70
        make = lambda: torch.empty((pages, page, heads, D), device="cuda", dtype=dtype)
    else:
        pages = (1 << 28) // (heads * D * size) + (1 if far == "more tokens" else -1)
        make = lambda: torch.empty((page, pages, heads, D), device="cuda", dtype=dtype).transpose(0, 1)
    width = 256 // page
    # both requests hold the first full page, pages - 1; the others are their own
    order = [pages - 1, 0, pages // 2 + 1, pages - 2, 5, pages - 3, 1, 2, pages - 4, pages // 3, 7, 8, 9, 10, 11, pages - 9, 13, 14]
    order += [x for x in range(20, 60)]
    table = np.array([order[:width], order[:1] + order[width:2 * width - 1]])
    used = sorted({int(p) for p in table.flat})
    near_table = np.array([[used.index(int(p)) for p in row] for row in table])
    g = torch.Generator(device="cuda").manual_seed(1)
    big, small = {}, {}
    for n in ("k", "v"):
        small[n + "_cache"] = torch.randn((len(used), page, heads, D), generator=g, device="cuda").to(dtype)
        big[n + "_cache"] = make()
        big[n + "_cache"].view(word)[used] = small[n + "_cache"].view(word)
        small[n + "_scale"] = big[n + "_scale"] = None
        if kind == "e4m3":
            small[n + "_scale"] = torch.randint(120, 126, (len(used), heads, page), generator=g, device="cuda", dtype=torch.uint8)
            big[n + "_scale"] = torch.full((pages, heads, page), 127, device="cuda", dtype=torch.uint8)
            big[n + "_scale"][used] = small[n + "_scale"]
    w = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
    for new in (1, 5, 40):
        q = torch.randn((2 * new, 32, D), generator=g, device="cuda").bfloat16()
        x = torch.randn((2 * new, heads, D), generator=g, device="cuda").bfloat16()
        a, b = (calls(c, t, new, q, x, w, [199, 170], page) for c, t in ((big, table), (small, near_table)))
        for n in b:
            assert torch.equal(a[n], b[n]), (new, n)
        assert torch.isfinite(b["s_lse"]).all() and torch.isfinite(b["g_lse"]).all()


@pytest.mark.parametrize("page", [1, 16])
def test_hints_change_roundings_only(page):
    """Hints too small, too large, and of more than 32 bits; every call twice, bit by bit."""
    new, total = [1, 5, 40, 0, 2], [1800, 1700, 900, 0, 640]
    pages, table, start = tables(new, total, page)
    table[1:, :600 // page] = table[0, :600 // page]
    c = fill(new_cache("bf16", pages, page, 2, 64), 8)
    q = torch.randn((48, 8, 64), device="cuda").bfloat16()
    cache = dict(k=values(c, "k"), v=values(c, "v"), table=table)
    a = (q, c["k_cache"], c["v_cache"], I32(table), I32(start), I32(total))
    want = osv.attention(N(q), cache, start, total, 0.125, 700, 50)
    for kw in ({}, dict(max_q_len=1), dict(max_q_len=40, max_kv_len=1800), dict(max_kv_len=3), dict(max_q_len=2 ** 40, max_kv_len=2 ** 33)):
        o, again = (sv.sv_paged_attention_sinks(*a, window=700, sinks=50, want_lse=True, **kw) for _ in range(2))
        within(o, want, 64, np.arange(48))
        assert torch.equal(o["out"], again["out"]) and torch.equal(o["lse"], again["lse"])
    groups, shared = [0, 3, 5], [600, 590]
    want = osv.attention(N(q), cache, start, total, 0.125, 0, 0, groups, shared)
    for kw in ({}, dict(max_q_len=1, max_group_len=1), dict(max_q_len=40, max_group_len=46, max_shared_len=600, max_own_len=1200),
               dict(max_shared_len=3, max_own_len=2), dict(max_q_len=2 ** 40, max_group_len=1),
               dict(max_q_len=1, max_group_len=2 ** 40, max_shared_len=2 ** 40, max_own_len=2 ** 40),
               dict(max_q_len=3, max_group_len=6, max_own_len=1200)):
        o, again = (sv.sv_paged_attention_shared(*a, I32(groups), I32(shared), want_lse=True, **kw) for _ in range(2))
        within(o, want, 64, np.arange(48))
        assert torch.equal(o["out"], again["out"]) and torch.equal(o["lse"], again["lse"])


def test_strided_rows_and_outputs():
    """Queries out of a fused projection, outputs in a wider buffer and head-major, a page table row for all requests."""
    new, total, D = [5, 40], [60, 64], 64
    pages, table, start = tables(new, total, 16)
    table[1] = table[0]
    c = fill(new_cache("bf16", pages, 16, 2, D), 1)
    fused = torch.randn((45, 12, D), device="cuda").bfloat16()
    q = fused[:, 2:10]
    k = (c["k_cache"], c["v_cache"])
    rest = (I32(start), I32(total))
    one_row = I32(table[:1]).expand(2, -1)
    sinks = lambda q, t, **kw: sv.sv_paged_attention_sinks(q, *k, t, *rest, window=9, sinks=3, **kw)["out"]
    shared = lambda q, t, **kw: sv.sv_paged_attention_shared(q, *k, t, *rest, I32([0, 2]), I32([20]), **kw)["out"]
    for call in (sinks, shared):
        want = call(q.contiguous(), I32(table))
        assert torch.equal(call(q, I32(table)), want) and torch.equal(call(q, one_row), want)
        wide = torch.full((45, 20, D), 5.0, device="cuda").bfloat16()
        assert torch.equal(call(q, I32(table), out=dict(out=wide[:, 8:16])), want)
        assert (wide[:, :8] == 5).all() and (wide[:, 16:] == 5).all()
        om = torch.empty((8, 45, D), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
        assert torch.equal(call(q.transpose(0, 1).contiguous().transpose(0, 1), I32(table), out=dict(out=om)), want)


@pytest.mark.parametrize("new,q_heads", [(1, 8), (40, 8)])
def test_few_of_a_billion_tokens(new, q_heads):
    """A context of 2^30 tokens less a few in a table of one repeated page: what a row sees with sinks and a window, and
    behind shared tokens that are nearly all, is what short contexts of the same tokens give."""
    page, D = 65536, 64
    c = fill(new_cache("bf16", 2, page, 2, D), 3)
    q = torch.randn((new, q_heads, D), device="cuda").bfloat16()
    n = (1 << 30) // page
    table = np.zeros((1, n), int)
    total = (1 << 30) - 1000
    a = (q, c["k_cache"], c["v_cache"])
    far = sv.sv_paged_attention_sinks(*a, I32(table), I32([0, new]), I32([total]), window=300, sinks=20, max_kv_len=total, want_lse=True)
    # the same tokens in two pages: the first ones, and the window at the same places of the second
    near = sv.sv_paged_attention_sinks(*a, I32(table[:, :2]), I32([0, new]), I32([2 * page - 1000]), window=300, sinks=20,
                                       max_kv_len=total, want_lse=True)
    assert torch.equal(far["out"], near["out"]) and torch.equal(far["lse"], near["lse"])
    # of 2^24 tokens none but those of the last page are held, most of them shared, the last 500 the request's own
    n, total = (1 << 24) // page, (1 << 24) - 1000
    table = np.full((1, n), -1)
    table[0, n - 1] = 1
    own = sv.sv_paged_attention_shared(*a, I32(table), I32([0, new]), I32([total]), I32([0, 1]), I32([total - 500]),
                                       max_q_len=new, max_group_len=new, max_shared_len=total, max_own_len=500, want_lse=True)
    plain = sv.sv_paged_attention(*a, I32([[1]]), I32([0, new]), I32([total - (n - 1) * page]), want_lse=True)
    # (both sum the same weights, each rounded to 2^-8 at most for the products, of about 64 thousand values near 1)
    assert torch.allclose(own["lse"], plain["lse"], atol=1e-4)
    assert torch.allclose(own["out"].float(), plain["out"].float(), rtol=2.0 ** -6, atol=2.0 ** -8)
