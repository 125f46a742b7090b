"""Caches whose tokens, not pages, are far apart: [page_size, num_pages, heads,
head_dim] seen as [num_pages, page_size, heads, head_dim].  The attention reads
16 tokens from one address with 32-bit offsets as long as they lie within 2^32
bytes (just so in one case here, just not in the other)."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from test_gpu_attn import call
from test_gpu_kv import I32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("more", [-1, 1])
def test_tokens_far_apart(kind, more):
    page, heads, D = 16, 8, 128
    size = 2 if kind == "bf16" else 1
    pages = (1 << 28) // (heads * D * size) + more  # a token's rows are about 2^28 bytes behind those of the one before
    dtype = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    table = np.array([[pages - 1, 0, pages // 2 + 1, pages - 2, 5], [pages - 3, 1, 2, pages - 4, pages // 3]])
    used = [int(p) for p in table.flat]
    g = torch.Generator(device="cuda").manual_seed(1)
    far, near = {}, {}
    for n in ("k", "v"):
        near[n + "_cache"] = torch.randn((len(used), page, heads, D), generator=g, device="cuda").to(dtype)
        far[n + "_cache"] = torch.empty((page, pages, heads, D), device="cuda", dtype=dtype).transpose(0, 1)
        far[n + "_cache"].view(torch.int8 if size == 1 else torch.int16)[used] = near[n + "_cache"].view(
            torch.int8 if size == 1 else torch.int16)
        near[n + "_scale"] = far[n + "_scale"] = None
        if kind == "e4m3":
            near[n + "_scale"] = torch.randint(120, 126, (len(used), heads, page), generator=g, device="cuda", dtype=torch.uint8)
            far[n + "_scale"] = torch.full((pages, heads, page), 127, device="cuda", dtype=torch.uint8)
            far[n + "_scale"][used] = near[n + "_scale"]
    both = (far, table), (near, np.arange(10).reshape(2, 5))
    for new in (3, 7, 50):
        start, total = [0, new, 2 * new], [79, 66]
        q = torch.randn((2 * new, 32, D), generator=g, device="cuda").bfloat16()
        x = torch.randn((2 * new, heads, D), generator=g, device="cuda").bfloat16()
        results = []
        for c, t in both:
            s = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
            sv.sv_kv_append(x, -x, c["k_cache"], c["v_cache"], I32(t), I32(start), I32(total), **s)
            o = call(q, c, t, start, total)
            o.update(sv.sv_kv_gather(c["k_cache"], c["v_cache"], I32(t), I32([0, 79, 145]), 145, **s))
            results.append(o)
        for n in ("out", "lse", "k", "v"):
            assert torch.equal(results[0][n], results[1][n]), (new, n)
        assert torch.isfinite(results[1]["lse"]).all()
