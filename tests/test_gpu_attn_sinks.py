"""sv_paged_attention_sinks on the GPU against the oracle; tolerances as derived
in test_gpu_attn.py."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import serve as osv
from test_gpu_attn import fill
from test_gpu_kv import I32, new_cache, tables, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

N = lambda x: x.double().cpu().numpy()


def within(o, w, D, rows):
    """Outputs and lse of these rows within the tolerance of test_gpu_attn.check."""
    out, lse = N(o["out"])[rows], N(o["lse"])[rows]
    want, wl, spread, size = (w[k][rows] for k in ("out", "lse", "spread", "size"))
    e = (D + 4) * 2.0 ** -24 * size + 2.0 ** -21
    tol = (2 * e[..., None] + 2 * 2.0 ** -8) * spread + np.abs(want) * 2.0 ** -8
    assert np.isfinite(out).all()
    assert (np.abs(out - want) <= tol).all(), (np.abs(out - want) - tol).max()
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(lse), empty) and (out[empty] == 0).all()
    assert (np.abs(lse - wl)[~empty] <= (e + np.abs(wl) * 2.0 ** -21)[~empty]).all()


def call(q, c, table, start, total, **kw):
    return sv.sv_paged_attention_sinks(q, c["k_cache"], c["v_cache"], I32(table), I32(start), I32(total),
                                       k_scale=c["k_scale"], v_scale=c["v_scale"], want_lse=True, **kw)


def oracle(q, c, table, start, total, scale, window, sinks):
    return osv.attention(N(q), dict(k=values(c, "k"), v=values(c, "v"), table=np.asarray(table)), start, total, scale, window,
                         sinks)


SHAPES = [  # new, lengths, page, kv heads, q heads, D
    ([1], [700], 16, 2, 8, 128),
    ([1, 1, 1], [5, 64, 333], 64, 1, 4, 128),
    ([5, 5, 5], [5, 200, 129], 16, 2, 8, 64),
    ([3, 0, 2], [260, 77, 2], 8, 2, 14, 64),
    ([2, 5], [33, 150], 1, 3, 3, 80),
    ([4, 1], [100, 301], 128, 2, 14, 96),
    ([7, 1], [90, 257], 32, 1, 2, 256),
    ([65, 130, 1], [65, 300, 205], 64, 1, 4, 128),
    ([70, 3], [300, 3], 16, 2, 6, 256),
    ([50], [360], 4, 1, 16, 112),
    ([140], [420], 64, 1, 1, 64),
]


@pytest.mark.parametrize("cache,order", [("bf16", "tokens"), ("e4m3", "heads")])
@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 4), (16, 4), (20, 33), (63, 64), (100, 129), (64, 0), (400, 4), (9, 900)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_sinks_match_the_oracle(cache, order, window, sinks, shape):
    new, total, page, heads, q_heads, D = SHAPES[shape]
    pages, table, start = tables(new, total, page, seed=shape)
    c = fill(new_cache(cache, pages, page, heads, D, order), shape)
    start = start + 2
    T = int(start[-1]) + 3
    q = torch.randn((T, q_heads, D), generator=torch.Generator(device="cuda").manual_seed(shape), device="cuda").bfloat16()
    want = oracle(q, c, table, start, total, D ** -0.5, window, sinks)
    for kw in ({}, dict(max_q_len=max(new), max_kv_len=max(total))):
        out = dict(out=torch.full_like(q, 9.0), lse=torch.full((T, q_heads), 9.0, device="cuda"))
        o = call(q, c, table, start, total, window=window, sinks=sinks, out=out, **kw)
        within(o, want, D, np.arange(start[0], start[-1]))
        for x in (o["out"], o["lse"]):  # rows of no request
            assert (x[:2] == 9.0).all() and (x[start[-1]:] == 9.0).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,window,sinks,total", [(1, 1000, 4, 5000), (3, 700, 200, 2500), (1, 3000, 70, 3200),
                                                    (40, 900, 5, 4000)])
def test_sinks_of_long_contexts(cache, new, window, sinks, total):
    """Windows that are divided into splits, the first of which holds the first tokens too."""
    news, totals = [new, 1], [total, total // 7]
    pages, table, start = tables(news, totals, 16)
    c = fill(new_cache(cache, pages, 16, 1, 64), 3)
    q = torch.randn((start[-1], 4, 64), device="cuda").bfloat16()
    o = call(q, c, table, start, totals, window=window, sinks=sinks, max_q_len=new, max_kv_len=total)
    within(o, oracle(q, c, table, start, totals, 0.125, window, sinks), 64, np.arange(start[-1]))


def test_degenerate_windows_are_the_plain_call():
    """No window, or one that reaches the first token: bit by bit what sv_paged_attention gives for the same plan; no
    sinks: its window's result but for roundings."""
    new, total = [5, 40, 1], [60, 200, 1500]
    pages, table, start = tables(new, total, 16)
    c = fill(new_cache("bf16", pages, 16, 2, 128), 1)
    q = torch.randn((46, 8, 128), device="cuda").bfloat16()
    a = (q, c["k_cache"], c["v_cache"], I32(table), I32(start), I32(total))
    for hints in ({}, dict(max_q_len=40, max_kv_len=1500)):
        plain = sv.sv_paged_attention(*a, want_lse=True, **hints)
        for window, sinks in ((0, 7), (0, 0), (10 ** 6, 3), (2 ** 40, 2 ** 40)):
            o = sv.sv_paged_attention_sinks(*a, window=window, sinks=sinks, want_lse=True, **hints)
            assert torch.equal(o["out"], plain["out"]) and torch.equal(o["lse"], plain["lse"])


@pytest.mark.parametrize("new", [3, 40])
def test_rows_that_see_nothing(new):
    """Lengths of zero and below the new rows' number; sinks or windows of absent pages alone."""
    page = 16
    table = np.array([[0, 1, 2, -1, -1], [-1, 3, 4, 5, 6], [7, 99, -1, -1, -5], [8, 9, 10, 11, 12]])
    total = [0, 75, 78, max(1, new - 2)]
    start = np.arange(5) * new
    c = fill(new_cache("bf16", 13, page, 2, 128), new)
    q = torch.randn((4 * new, 4, 128), device="cuda").bfloat16()
    for window, sinks in ((12, 5), (1, 16), (30, 1)):
        o = call(q, c, table, start, total, window=window, sinks=sinks)
        want = oracle(q, c, table, start, total, 128 ** -0.5, window, sinks)
        assert np.isneginf(want["lse"][:new]).all()
        within(o, want, 128, np.arange(4 * new))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,window,sinks", [(1, 20, 5), (5, 64, 33), (40, 50, 7), (140, 70, 10)])
def test_what_is_between_sinks_and_window_has_no_influence(cache, new, window, sinks):
    """NaN, infinities and extremes in tokens that no row sees, in the pieces next to the seen ones too, change no bit."""
    page, D, total = 16, 128, 500
    pages, table, start = tables([new], [total], page, spare=3)
    c = fill(new_cache(cache, pages, page, 1, D), 5)
    q = torch.randn((new, 4, D), device="cuda").bfloat16()
    clean = call(q, c, table, start, [total], window=window, sinks=sinks)
    within(clean, oracle(q, c, table, start, [total], D ** -0.5, window, sinks), D, np.arange(new))
    bad = [float("nan"), float("inf"), float("-inf"), 3e38] if cache == "bf16" else [float("nan")]
    seen = {(int(table[0, j // page]), j % page) for j in range(total) if j < sinks or j > total - new - window}
    i = 0
    for n in ("k", "v"):
        for p in range(pages):
            for s in range(page):
                if (p, s) not in seen:
                    c[n + "_cache"][p, s] = torch.full((1, D), bad[i % len(bad)], device="cuda").to(c[n + "_cache"].dtype)
                    if c[n + "_scale"] is not None:
                        c[n + "_scale"][p, :, s] = [255, 120, 254][i % 3]
                    i += 1
    o = call(q, c, table, start, [total], window=window, sinks=sinks)
    assert torch.equal(o["out"], clean["out"]) and torch.equal(o["lse"], clean["lse"])


def test_sinks_seen_by_some_rows_only():
    """A token that is not finite and that later rows do not see spoils those that do, and no other bit."""
    new, total, window = 40, 100, 8
    pages, table, start = tables([new], [total], 16)
    c = fill(new_cache("bf16", pages, 16, 1, 64), 2)
    q = torch.randn((new, 2, 64), device="cuda").bfloat16()
    clean = call(q, c, table, start, [total], window=window, sinks=3)
    c["v_cache"][table[0, 70 // 16], 70 % 16] = float("inf")
    o = call(q, c, table, start, [total], window=window, sinks=3)
    sees = torch.tensor([60 + i >= 70 > 60 + i - window for i in range(new)], device="cuda")
    assert torch.equal(o["out"][~sees], clean["out"][~sees]) and torch.equal(o["lse"][~sees], clean["lse"][~sees])
    assert not torch.isfinite(o["out"][sees].float()).any() and sees.sum() == window
    c["k_cache"][table[0, 0], 2] = float("nan")  # a first token: every row sees it
    assert torch.isnan(call(q, c, table, start, [total], window=window, sinks=3)["lse"]).all()


def test_sinks_captured_and_on_two_streams():
    def make(seed):
        new, total = (3, 1, 5), (900, 40, 2333)
        pages, table, start = tables(new, total, 16, seed=seed)
        c = fill(new_cache("bf16", pages, 16, 2, 128), seed)
        q = torch.randn((9, 8, 128), device="cuda").bfloat16()
        return dict(q=q, c=c, a=(c["k_cache"], c["v_cache"], I32(table), I32(start), I32(total)))

    run = lambda s: sv.sv_paged_attention_sinks(s["q"], *s["a"], window=600, sinks=40, max_q_len=5, max_kv_len=2333, want_lse=True)
    ss = [make(k) for k in (1, 2)]
    for s in ss:
        run(s)
    torch.cuda.synchronize()
    graphs = []
    for s in ss:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(s)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in ss]
    for rep in range(4):
        for s in ss:
            s["q"].copy_(torch.randn(s["q"].shape, device="cuda"))
            s["a"][4].sub_(7 * rep)
        want = [{k: v.clone() for k, v in run(s).items()} for s in ss]
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager = []
        for s, st in zip(ss, streams):
            with torch.cuda.stream(st):
                eager.append(run(s))
        torch.cuda.synchronize()
        for w, (_, out), e in zip(want, graphs, eager):
            for k in w:
                assert torch.equal(out[k], w[k]) and torch.equal(e[k], w[k]), (rep, k)


def test_scratch_of_the_caller():
    new, total = [2, 1], [9000, 100]
    pages, table, start = tables(new, total, 64)
    c = fill(new_cache("bf16", pages, 64, 1, 64), 4)
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    kw = dict(window=4000, sinks=4, max_q_len=2, max_kv_len=9000)
    want = call(q, c, table, start, total, **kw)
    size = sv.sv_paged_attention_sinks_workspace_size(2, 3, 4, 1, 64, 2, 9000, 4000, 4)
    assert 256 < size < sv.sv_paged_attention_workspace_size(2, 3, 4, 1, 64, 2, 9000)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    got = call(q, c, table, start, total, workspace=ws[:size], **kw)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"]) and (ws[size:] == 255).all()
    with pytest.raises(RuntimeError, match="workspace"):
        call(q, c, table, start, total, workspace=ws[:size - 1], **kw)
    for bad in (dict(window=-1, sinks=4), dict(window=4, sinks=-1)):
        with pytest.raises(RuntimeError, match="invalid argument"):
            call(q, c, table, start, total, workspace=ws[:size], **bad)
