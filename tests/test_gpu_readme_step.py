"""The loop of README.md (one layer's share of a verification step), run as it
stands there for several steps."""
import os
import re

import pytest
import torch

import draft_token_verification_spec_amd as sv
from test_gpu_attn import check, fill
from test_gpu_kv import I32, new_cache

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def loop():
    """(setup, step): the indented block's lines up to the frequencies, and those behind them."""
    block = re.search(r"((?:^    .*\n|^\n)*^    .*sv_paged_attention(?:.*\n)(?:^    .*\n)*)", open(README).read(), re.M).group(1)
    lines = [x[4:] for x in block.strip("\n").split("\n")]
    at = next(i for i, x in enumerate(lines) if "sv_rope_frequencies" in x) + 1
    return "\n".join(lines[:at]), "\n".join(lines[at:])


def test_readme_step():
    setup, step = loop()
    B, K, Hq, H, D, page = 3, 4, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    c = fill(new_cache("bf16", 30, page, H, D), 1)
    table = torch.randperm(30, generator=g, device="cuda").int().view(B, 10)
    ns = dict(k_cache=c["k_cache"], v_cache=c["v_cache"], page_table=table, K=K,
              query_start=I32([0, K + 1, 2 * (K + 1), 3 * (K + 1)]), kv_len=I32([0, 0, 0]))
    exec(setup, ns)
    assert ns["freq"].shape == (D // 2,)
    # frequencies whose mscale is not 1: the step has to pass it on
    ns["freq"], ns["mscale"] = sv.sv_rope_frequencies(D, scaling="ramp", factor=8.0, original_len=64.0, device="cuda")
    assert ns["mscale"] != 1.0
    kept = [[] for _ in range(B)]  # (key, value) of each token that a request has kept
    for accept in ([4, 0, 2], [0, 0, 4], [1, 3, 2], [4, 4, 0]):
        q, k, v = (torch.randn((B * (K + 1), h, D), generator=g, device="cuda").bfloat16() for h in (Hq, H, H))
        ns.update(q=q, k=k, v=v, accept_len=I32(accept))
        before = [len(x) for x in kept]
        exec(step, ns)
        places = torch.tensor([n + i for n in before for i in range(K + 1)], device="cuda")
        turned = [sv.sv_rope(x, places, ns["freq"], mscale=ns["mscale"]) for x in (q, k)]
        assert torch.equal(ns["q"], turned[0])
        total = [n + K + 1 for n in before]
        check(dict(out=ns["o"], lse=sv.sv_paged_attention(turned[0], ns["k_cache"], ns["v_cache"], table, ns["query_start"],
                                                         I32(total), want_lse=True)["lse"]),
              turned[0], c, table.cpu().numpy(), ns["query_start"].tolist(), total, D ** -0.5)
        for b in range(B):
            first = b * (K + 1)
            kept[b] += [(turned[1][first + i], v[first + i]) for i in range(1 + accept[b])]
        # the cache holds what was kept, and the lengths say so
        assert ns["kv_len"].tolist() == [len(x) for x in kept]
        start = I32([0] + [sum(len(x) for x in kept[:b + 1]) for b in range(B)])
        back = sv.sv_kv_gather(ns["k_cache"], ns["v_cache"], table, start, int(start[-1]))
        flat = [x for b in range(B) for x in kept[b]]
        assert torch.equal(back["k"], torch.stack([x[0] for x in flat]))
        assert torch.equal(back["v"], torch.stack([x[1] for x in flat]))
