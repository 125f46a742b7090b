"""The cache and attention calls as a verification step uses them: several steps
of append, attention and sv_spec_verify with drafts rejected in between, the
same calls captured and replayed, on two streams at once, and with a scratch of
the caller's."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import attn as oa
from oracle import verify as ov
from test_gpu_attn import call, check, fill
from test_gpu_kv import I32, new_cache, tables, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_verification_steps_with_rejected_drafts(kind):
    """A one-layer target over 5 requests: every step appends K + 1 tokens, attends, verifies, and keeps the cache up
    to the accepted drafts by lengths alone; what the rejected drafts left is overwritten.  After each step the cache
    holds, for every request, the turned keys and values of exactly its accepted tokens."""
    B, K, Hq, H, D, V, page = 5, 4, 8, 2, 64, 512, 16
    g = torch.Generator(device="cuda").manual_seed(11)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    embed = rn(V, 96)
    wq, wk, wv = (rn(96, h * D) / 96 ** 0.5 for h in (Hq, H, H))
    head = rn(Hq * D, V) / (Hq * D) ** 0.5 * 6
    f, m = sv.sv_rope_frequencies(D, device="cuda")
    rng = np.random.default_rng(3)
    history = [rng.integers(0, V, n).tolist() for n in (1, 7, 16, 33, 2)]  # tokens with their keys in the cache
    last = rng.integers(0, V, B).tolist()                                  # the last token emitted, not yet there
    table = I32(rng.permutation(B * 6).reshape(B, 6))
    c = new_cache(kind, B * 6, page, H, D)
    cache = (c["k_cache"], c["v_cache"], table)
    s = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    rows = lambda tokens, w, h: (embed[torch.tensor(tokens, device="cuda")] @ w).view(-1, h, D).bfloat16()

    flat = sum(history, [])
    start = np.cumsum([0] + [len(t) for t in history])
    sv.sv_kv_append(rows(flat, wk, H), rows(flat, wv, H), *cache, I32(start), I32([len(t) for t in history]), freq=f, **s)
    rejected = 0
    for step in range(5):
        drafts = rng.integers(0, V, (B, K)).astype(np.int32)
        new = [[last[b]] + drafts[b].tolist() for b in range(B)]
        flat = sum(new, [])
        kv_len = I32([len(history[b]) + K + 1 for b in range(B)])
        start = I32(np.arange(B + 1) * (K + 1))
        q = rows(flat, wq, Hq)
        q = sv.sv_kv_append(rows(flat, wk, H), rows(flat, wv, H), *cache, start, kv_len, q=q, freq=f, **s)["q"]
        o = sv.sv_paged_attention(q, *cache, start, kv_len, max_q_len=K + 1, max_kv_len=96, want_lse=True, **s)
        check(o, q, c, table.cpu().numpy(), (np.arange(B + 1) * (K + 1)).tolist(), kv_len.tolist(), D ** -0.5)
        logits = (o["out"].float().view(-1, Hq * D) @ head).contiguous()
        # half of the drafts are made what greedy verification would accept
        tgt = logits.view(B, K + 1, V).argmax(-1).cpu().numpy()
        keep = rng.integers(0, K + 1, B)
        for b in range(B):
            drafts[b, :keep[b]] = tgt[b, :keep[b]] if keep[b] else drafts[b, :0]
        nd = I32([K] * B)
        zero, u = torch.zeros(B, device="cuda"), torch.rand((B, K), generator=g, device="cuda")
        first = torch.arange(B, device="cuda") * (K + 1)
        r = sv.sv_spec_verify(logits, first, logits, first, nd, I32(drafts), zero, u, u[:, 0].contiguous(),
                              u[:, 1].contiguous(), max_k=K)
        acc, tok = r["accept_len"].cpu().numpy(), r["out_tokens"].cpu().numpy()
        for b in range(B):
            want = next((i for i in range(K) if drafts[b, i] != tgt[b, i]), K)
            assert acc[b] == want and tok[b, want] == tgt[b, want]
            # (the cache holds the keys of the tokens that were run, `new`: only those can be kept)
            kept = next((i for i in range(acc[b]) if drafts[b, i] != new[b][1 + i]), acc[b])
            rejected += K - kept
            history[b] += new[b][: 1 + kept]
            last[b] = int(tok[b, kept])
        # what the cache stands for now, by the lengths that the next step starts from
        lengths = [len(t) for t in history]
        start = np.cumsum([0] + lengths)
        back = sv.sv_kv_gather(*cache, I32(start), int(start[-1]), dtype=torch.float32, **s)
        flat = sum(history, [])
        place = np.concatenate([np.arange(n) for n in lengths])
        kx, vx = rows(flat, wk, H), rows(flat, wv, H)
        n = lambda t: t.double().cpu().numpy()
        turned = oa.rope(n(kx), place, n(f), "half", m)
        err = np.abs(n(kx)).max(-1, keepdims=True) * 2.0 ** -20  # the rotation's (see test_gpu_rope), doubled
        step_of = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}[kind]
        floor = 0 if kind == "bf16" else np.abs(turned).max(-1, keepdims=True) / 224 * 2.0 ** -10
        assert (np.abs(n(back["k"]) - turned) <= (err + np.maximum(np.abs(turned) * step_of, floor)) * 1.0625).all()
        if kind == "bf16":
            assert np.array_equal(n(back["v"]), n(vx))
        else:
            codes, e = oa.quantise(n(vx))
            assert np.array_equal(n(back["v"]), oa.e4m3_values()[codes] * 2.0 ** e[..., None])
    assert rejected > 10


def step_inputs(seed, kind="bf16", new=(3, 1, 5), total=(900, 40, 333)):
    pages, table, start = tables(new, total, 16, seed=seed)
    c = fill(new_cache(kind, pages, 16, 2, 128), seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((start[-1], 12, 128), generator=g, device="cuda").bfloat16()
    f, _ = sv.sv_rope_frequencies(128, device="cuda")
    return dict(c=c, qkv=qkv, f=f, table=I32(table), start=I32(start), total=I32(total), max_q=max(new), max_kv=max(total))


def run_step(s):
    q, k, v = s["qkv"].split([8, 2, 2], 1)
    c = s["c"]
    a = (c["k_cache"], c["v_cache"], s["table"])
    sc = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    q = sv.sv_kv_append(k, v, *a, s["start"], s["total"], q=q, freq=s["f"], **sc)["q"]
    o = sv.sv_paged_attention(q, *a, s["start"], s["total"], max_q_len=s["max_q"], max_kv_len=s["max_kv"], want_lse=True, **sc)
    back = sv.sv_kv_gather(*a, s["start"], q.shape[0], kv_begin=s["total"] - s["start"].diff(), **sc)
    turned = sv.sv_rope(o["out"], torch.arange(q.shape[0], device="cuda"), s["f"], backward=True)
    return dict(q=q, out=o["out"], lse=o["lse"], k=back["k"], v=back["v"], turned=turned)


@pytest.mark.parametrize("kind,new,total", [("bf16", (3, 1, 5), (900, 40, 333)), ("e4m3", (90, 2), (1500, 9))])
def test_graph_replays_match_eager(kind, new, total):
    """Captured calls replayed with other inputs in place, among eager calls: two graphs that live at the same time."""
    ss = [step_inputs(k, kind, new, total) for k in (1, 2)]
    for s in ss:
        run_step(s)
    torch.cuda.synchronize()
    graphs = []
    for s in ss:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run_step(s)
        graphs.append((g, out))
    for rep in range(4):
        for s, (g, out) in zip(ss, graphs):
            s["qkv"].copy_(torch.randn(s["qkv"].shape, device="cuda"))
            s["total"].sub_(1 + rep)  # shorter contexts: other splits are live
            g.replay()
            other = run_step(ss[0] if s is ss[1] else ss[1])  # eager work on another cache in between
            torch.cuda.synchronize()
            got = {k: v.clone() for k, v in out.items()}
            want = run_step(s)
            for k in want:
                assert torch.equal(got[k], want[k]), (rep, k)
            assert not torch.isnan(other["lse"]).any()  # (-inf where the shortened context leaves nothing)


def test_two_streams_at_once():
    ss = [step_inputs(k, total=(3000, 40, 2000)) for k in (5, 6)]
    want = [{k: v.clone() for k, v in run_step(s).items()} for s in ss]
    streams = [torch.cuda.Stream() for _ in ss]
    torch.cuda.synchronize()
    for rep in range(10):
        got = []
        for s, st in zip(ss, streams):
            with torch.cuda.stream(st):
                got.append(run_step(s))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            for k in y:
                assert torch.equal(x[k], y[k]), (rep, k)


def test_callers_scratch():
    """What a scratch holds does not matter, nothing beyond its stated size is written, and one too small is refused."""
    new, total = [2, 1], [5000, 100]
    pages, table, start = tables(new, total, 64)
    c = fill(new_cache("bf16", pages, 64, 1, 64), 4)
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    want = call(q, c, table, start, total, max_q_len=2, max_kv_len=5000)
    size = sv.sv_paged_attention_workspace_size(2, 3, 4, 1, 64, 2, 5000)
    assert size > 256  # the long context is split
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got = call(q, c, table, start, total, max_q_len=2, max_kv_len=5000, workspace=ws[:size])
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
        assert (ws[size:] == 255).all()
    with pytest.raises(RuntimeError, match="workspace"):
        call(q, c, table, start, total, max_q_len=2, max_kv_len=5000, workspace=ws[:size - 1])
    with pytest.raises(TypeError):
        call(q, c, table, start, total, workspace=ws.float())


def test_values_of_the_cache_are_left_alone():
    """Attention and gather write nothing of the cache; append nothing but its slots (see test_gpu_kv)."""
    s = step_inputs(9, "e4m3", (20, 1), (60, 700))
    run_step(s)
    before = {k: v.clone().view(torch.uint8) for k, v in s["c"].items()}
    run_step(s)  # the same rows into the same slots
    for k, v in s["c"].items():
        assert torch.equal(v.view(torch.uint8), before[k]), k
