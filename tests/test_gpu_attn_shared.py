"""sv_paged_attention_shared on the GPU against the oracle; tolerances as derived
in test_gpu_attn.py (a row's parts are joined in binary32, a few roundings of
2^-24 more, far below the second 2^-8 there)."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import serve as osv
from test_gpu_attn import fill
from test_gpu_attn_sinks import N, within
from test_gpu_kv import I32, new_cache, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


def batch(kind, new, total, groups, shared, page, heads, q_heads, D, order="tokens", seed=0, copies=True):
    """Requests whose rows of the page table agree in the full shared pages; a page shared in part is copied."""
    rng = np.random.default_rng(seed)
    B, width = len(new), max(-(-max(t, 1) // page) for t in list(total) + list(shared)) + 1
    order_of = iter(rng.permutation(B * width + 3))
    table = np.full((B, width), -1)
    same = []
    for b in range(B):
        g = next((i for i in range(len(shared)) if groups[i] <= b < groups[i + 1]), None)
        n = 0 if g is None else max(shared[g], 0)
        first = b if g is None else groups[g]
        hold = max(-(-max(total[b], 0) // page), -(-n // page) if b == first else 0)
        for i in range(hold):
            if b != first and (i + 1) * page <= n:
                table[b, i] = table[first, i]
                continue
            table[b, i] = next(order_of)
            if b != first and i * page < n:
                same.append((int(table[first, i]), int(table[b, i]), n - i * page))
    c = fill(new_cache(kind, B * width + 3, page, heads, D, order), seed)
    if copies:
        for src, to, n in same:
            for x in ("k", "v"):
                c[x + "_cache"].view(torch.uint8)[to, :n] = c[x + "_cache"].view(torch.uint8)[src, :n]
                if c[x + "_scale"] is not None:
                    c[x + "_scale"][to, :, :n] = c[x + "_scale"][src, :, :n]
    start = np.cumsum([0] + list(new))
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((int(start[-1]), q_heads, D), generator=g, device="cuda").bfloat16()
    return dict(q=q, c=c, table=table, start=start, total=list(total), groups=list(groups), shared=list(shared))


def call(s, q=None, start=None, **kw):
    c = s["c"]
    return sv.sv_paged_attention_shared(s["q"] if q is None else q, c["k_cache"], c["v_cache"], I32(s["table"]),
                                        I32(s["start"] if start is None else start), I32(s["total"]), I32(s["groups"]),
                                        I32(s["shared"]), k_scale=c["k_scale"], v_scale=c["v_scale"], want_lse=True, **kw)


def oracle(s, scale, q=None, start=None):
    c = dict(k=values(s["c"], "k"), v=values(s["c"], "v"), table=s["table"])
    return osv.attention(N(s["q"] if q is None else q), c, s["start"] if start is None else start, s["total"], scale, 0, 0,
                         s["groups"], s["shared"])


def hints(s):
    new = np.diff(s["start"])
    of = [max(0, next((s["shared"][i] for i in range(len(s["shared"])) if s["groups"][i] <= b < s["groups"][i + 1]), 0))
          for b in range(len(new))]
    return dict(max_q_len=int(max(new)), max_shared_len=max(s["shared"] + [1]),
                max_group_len=max([int(s["start"][b] - s["start"][a]) for a, b in zip(s["groups"], s["groups"][1:])] + [1]),
                max_own_len=max(1, max(t - n for t, n in zip(s["total"], of))))


SHAPES = [  # new, lengths, group starts, shared, page, kv heads, q heads, D
    ([1] * 4, [110, 103, 140, 101], [0, 4], [100], 16, 2, 8, 128),
    ([1] * 20, list(range(301, 321)), [0, 20], [300], 16, 1, 4, 128),
    ([5] * 30, [200 + 7 * i for i in range(30)], [0, 30], [190], 16, 2, 4, 64),
    ([3, 0, 2, 1, 1, 4], [90, 64, 72, 41, 300, 44], [1, 3, 5], [64, 40], 8, 2, 8, 64),
    ([2] * 7, [40, 41, 70, 33, 34, 35, 36], [0, 3, 3, 7], [38, 5, 31], 1, 3, 3, 80),
    ([4, 1, 9], [150, 131, 150], [0, 3], [128], 128, 2, 14, 96),
    ([7, 1, 6], [90, 257, 88], [0, 3], [80], 32, 1, 2, 256),
    ([65, 30, 1], [165, 140, 105], [0, 3], [100], 64, 1, 4, 128),
    ([70, 3], [300, 203], [0, 2], [199], 16, 2, 6, 256),
    ([40, 1, 50], [60, 15, 64], [0, 3], [14], 16, 1, 8, 112),
    ([1] * 9, [17 + i for i in range(9)], [0, 2, 5, 9], [16, 0, -3], 16, 1, 16, 64),
]


@pytest.mark.parametrize("cache,order", [("bf16", "tokens"), ("e4m3", "heads")])
@pytest.mark.parametrize("hinted", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shared_matches_the_oracle(cache, order, hinted, shape):
    new, total, groups, shared, page, heads, q_heads, D = SHAPES[shape]
    s = batch(cache, new, total, groups, shared, page, heads, q_heads, D, order, shape)
    start = s["start"] + 2
    T = int(start[-1]) + 3
    q = torch.zeros((T, q_heads, D), device="cuda", dtype=torch.bfloat16)
    q[2:start[-1]] = s["q"]
    out = dict(out=torch.full_like(q, 9.0), lse=torch.full((T, q_heads), 9.0, device="cuda"))
    o = call(s, q, start, out=out, **(hints(s) if hinted else {}))
    within(o, oracle(s, D ** -0.5, q, start), D, np.arange(2, start[-1]))
    for x in (o["out"], o["lse"]):  # rows of no request
        assert (x[:2] == 9.0).all() and (x[start[-1]:] == 9.0).all()
    plain = sv.sv_paged_attention(q, s["c"]["k_cache"], s["c"]["v_cache"], I32(s["table"]), I32(start), I32(total),
                                  k_scale=s["c"]["k_scale"], v_scale=s["c"]["v_scale"], want_lse=True)
    assert torch.allclose(o["lse"][2:start[-1]], plain["lse"][2:start[-1]], atol=1e-4)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,shared,own", [(1, 5000, 40), (1, 700, 3000), (5, 2100, 1500), (40, 1300, 100)])
def test_shared_long(cache, new, shared, own):
    """Both parts divided into several splits."""
    s = batch(cache, [new] * 3, [shared + own - 7 * i for i in range(3)], [0, 3], [shared], 16, 1, 4, 64)
    o = call(s, **hints(s))
    within(o, oracle(s, 0.125), 64, np.arange(3 * new))


def test_rows_of_the_shared_tokens_themselves():
    """New tokens that lie among the shared ones see those up to their own places; lengths below the rows' number, of zero
    and below zero see nothing; a request that holds the shared tokens alone sees those."""
    for q_heads in (2, 32):
        s = batch("bf16", [3, 4, 2, 1, 5, 1], [30, 26, 20, 1, 3, 24], [0, 6], [24], 8, 2, q_heads, 64, seed=q_heads)
        s["total"][3] = 0
        want = oracle(s, 0.125)
        assert np.isneginf(want["lse"][9]).all() and np.isneginf(want["lse"][10:12]).all()
        for kw in ({}, hints(s)):
            within(call(s, **kw), want, 64, np.arange(16))
        s["total"][2] = -5
        within(call(s), oracle(s, 0.125), 64, np.arange(16))


def test_first_request_without_rows_or_length():
    """The shared pages are those of the first request's row, whatever else is known of it."""
    s = batch("bf16", [0, 2, 2], [40, 50, 44], [0, 3], [40], 16, 1, 4, 64)
    s["total"][0] = 0
    within(call(s), oracle(s, 0.125), 64, np.arange(4))
    s["table"][0, 1] = -1  # a shared page that is absent is so for all
    within(call(s), oracle(s, 0.125), 64, np.arange(4))
    s["table"][0] = -1
    s["total"] = [0, 40, 41]
    want = oracle(s, 0.125)
    assert np.isneginf(want["lse"][:3]).all()
    within(call(s), want, 64, np.arange(4))


@pytest.mark.parametrize("new,q_heads", [(1, 4), (5, 4), (40, 4)])
def test_shared_ignores_what_it_does_not_see(new, q_heads):
    """What the other requests hold at the shared places, tokens behind the ends and unused pages: no bit changes."""
    s = batch("bf16", [new] * 3, [90 + new, 77 + new, 70 + new], [0, 3], [70], 16, 1, q_heads, 128)
    clean = call(s)
    within(clean, oracle(s, 128 ** -0.5), 128, np.arange(3 * new))
    seen = set()
    for b in range(3):
        seen |= {(int(s["table"][0 if j < 70 else b, j // 16]), j % 16) for j in range(s["total"][b])}
    bad, i = [float("nan"), float("inf"), float("-inf"), 3e38], 0
    for x in ("k_cache", "v_cache"):
        for p in range(s["c"][x].shape[0]):
            for slot in range(16):
                if (p, slot) not in seen:
                    s["c"][x][p, slot] = bad[i % 4]
                    i += 1
    o = call(s)
    assert torch.equal(o["out"], clean["out"]) and torch.equal(o["lse"], clean["lse"])
    # a shared token that is not finite is seen by all, an own one by its request
    at = (int(s["table"][1, 76 // 16]), 76 % 16)
    s["c"]["k_cache"][at] = float("nan")
    o = call(s)
    mine = slice(new, 2 * new)
    assert torch.isnan(o["lse"][mine]).all()
    assert torch.equal(o["lse"][:new], clean["lse"][:new]) and torch.equal(o["out"][2 * new:], clean["out"][2 * new:])
    s["c"]["v_cache"][int(s["table"][0, 1]), 3] = float("inf")
    assert not torch.isfinite(call(s)["out"].float()).any()


def test_no_groups_and_groups_of_one():
    s = batch("bf16", [3, 1, 20], [50, 9, 333], [0], [], 16, 2, 8, 128)
    c = s["c"]
    plain = sv.sv_paged_attention(s["q"], c["k_cache"], c["v_cache"], I32(s["table"]), I32(s["start"]), I32(s["total"]), want_lse=True)
    o = call(s)
    assert torch.equal(o["out"], plain["out"]) and torch.equal(o["lse"], plain["lse"])
    s["groups"], s["shared"] = [0, 1, 2, 3], [33, 9, 200]
    within(call(s, **hints(s)), oracle(s, 128 ** -0.5), 128, np.arange(24))


def test_bad_groups_touch_nothing_else():
    """Group starts outside the batch or descending, lengths beyond the table: no memory beyond the arrays is read, and
    requests of no group are as ever."""
    s = batch("bf16", [2, 1, 3], [50, 9, 61], [0, 2], [8], 16, 1, 4, 64)
    s["shared"] = [2 ** 31 - 1]
    o = call(s)
    within(o, oracle(dict(s, shared=[s["table"].shape[1] * 16]), 0.125), 64, np.arange(6))
    for groups in ([-3, 2], [0, 9], [2, 1]):
        s["groups"], s["shared"] = groups, [8]
        o = call(s)
        assert o["out"].shape == (6, 4, 64)


def test_shared_captured_and_on_two_streams():
    ss = [batch("bf16", [2] * 12, [400 + 30 * i for i in range(12)], [0, 7, 12], [390, 500], 16, 2, 8, 128, seed=k) for k in (1, 2)]
    for s in ss:
        s["a"] = (s["c"]["k_cache"], s["c"]["v_cache"], I32(s["table"]), I32(s["start"]), I32(s["total"]), I32(s["groups"]), I32(s["shared"]))
        s["h"] = hints(s)
    run = lambda s: sv.sv_paged_attention_shared(s["q"], *s["a"], want_lse=True, **s["h"])
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
            s["a"][4].sub_(9 * rep)  # lengths, and what is shared
            s["a"][6].sub_(33 * rep)
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
    s = batch("bf16", [2, 1, 1], [3000, 2100, 2050], [0, 3], [2000], 64, 1, 4, 64)
    want = call(s, **hints(s))
    h = hints(s)
    size = sv.sv_paged_attention_shared_workspace_size(3, 4, 1, 4, 1, 64, h["max_q_len"], h["max_group_len"],
                                                       h["max_shared_len"], h["max_own_len"])
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    got = call(s, workspace=ws[:size], **h)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"]) and (ws[size:] == 255).all()
    with pytest.raises(RuntimeError, match="workspace"):
        call(s, workspace=ws[:size - 1], **h)
