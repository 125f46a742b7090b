"""sv_paged_attention over keys that are infinite: a score of -infinity is a
weight of zero, one of +infinity makes its row NaN, at every head size (16 to
256, which the kernels pad to 64, 128 or 256) and through every kernel.

A token whose score is -infinity and one whose score is finite and far below all
others have weights of zero alike and change nothing else, so the two calls are
compared bit for bit."""
import pytest
import torch

from test_gpu_attn import call, fill
from test_gpu_kv import new_cache, tables

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


@pytest.mark.parametrize("page", [4, 16, 64])
@pytest.mark.parametrize("new,total", [(1, 70), (7, 70), (40, 150)])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 176, 240, 256])
def test_attention_of_infinite_keys(D, new, total, page):
    pages, table, start = tables([new], [total], page, seed=D)
    c = fill(new_cache("bf16", pages, page, 1, D), D)
    g = torch.Generator(device="cuda").manual_seed(D + new)
    q = torch.randn((new, 4, D), generator=g, device="cuda").bfloat16()
    for token, channel in ((3, D - 1), (total - new, D - 6), (40, 0)):
        q[..., channel] = 1.0
        at = int(table[0, token // page]), token % page, 0, channel
        keep = float(c["k_cache"][at])
        c["k_cache"][at] = -2.0 ** 100
        want = call(q, c, table, start, [total])
        assert torch.isfinite(want["out"]).all() and torch.isfinite(want["lse"]).all()
        c["k_cache"][at] = float("-inf")
        got = call(q, c, table, start, [total])
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
        q[:, 1, channel] = -1.0  # the same token's score is +infinity for this head
        got = call(q, c, table, start, [total])
        assert torch.isnan(got["out"][:, 1]).all() and torch.isnan(got["lse"][:, 1]).all()
        others = [0, 2, 3]
        assert torch.equal(got["out"][:, others], want["out"][:, others])
        assert torch.equal(got["lse"][:, others], want["lse"][:, others])
        c["k_cache"][at] = keep


@pytest.mark.parametrize("new,total", [(1, 37), (9, 1500), (50, 90)])
@pytest.mark.parametrize("D", [80, 128])
def test_attention_of_scores_of_minus_infinity_alone(D, new, total):
    """A row without any weight gets what a row that sees nothing gets."""
    pages, table, start = tables([new], [total], 16)
    c = fill(new_cache("bf16", pages, 16, 1, D), 1)
    c["k_cache"][..., D - 1] = float("-inf")
    q = torch.randn((new, 3, D), device="cuda").bfloat16()
    q[..., D - 1] = 0.5
    o = call(q, c, table, start, [total], max_kv_len=total)
    assert (o["out"] == 0).all() and torch.isneginf(o["lse"]).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [4, 16, 64])
@pytest.mark.parametrize("new,q_heads,total", [(1, 4, 37), (7, 4, 1500), (40, 4, 175)])
@pytest.mark.parametrize("D", [48, 80, 240])
def test_padded_heads_ignore_what_they_do_not_see(D, new, q_heads, total, page, cache):
    """NaN and infinities behind the end, before the window and on other pages change nothing at padded sizes either."""
    window = 30
    pages, table, start = tables([new], [total], page, spare=3, seed=D)
    c = fill(new_cache(cache, pages, page, 1, D), D)
    q = torch.randn((new, q_heads, D), device="cuda").bfloat16()
    kw = dict(window=window, max_q_len=new, max_kv_len=total)
    clean = call(q, c, table, start, [total], **kw)
    assert torch.isfinite(clean["out"]).all()
    seen = torch.zeros((pages, page), dtype=torch.bool)
    for j in range(max(0, total - new - window + 1), total):
        seen[int(table[0, j // page]), j % page] = True
    hidden = (~seen).nonzero().cuda()
    for bad in (float("nan"), float("inf"), float("-inf")) if cache == "bf16" else (float("nan"),):
        for n in ("k", "v"):
            x = c[n + "_cache"]
            some = torch.full((len(hidden), 1, D), bad, device="cuda").to(x.dtype)
            bits = torch.int16 if cache == "bf16" else torch.uint8
            x.view(bits)[hidden[:, 0], hidden[:, 1]] = some.view(bits)
        got = call(q, c, table, start, [total], **kw)
        assert torch.equal(got["out"], clean["out"]) and torch.equal(got["lse"], clean["lse"])
