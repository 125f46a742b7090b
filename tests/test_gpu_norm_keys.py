"""Stored keys of sv_kv_append_normed: formed in binary64 from rows of any finite
size, and rounded to the cache's type once (bf16: by way of binary32).

The kernel's binary64 differs from the oracle's by some 2^-45 of a pair's size
(the root's one step of Newton's method from a binary32 estimate).  Of the 25
thousand keys of a case one lies that near to the middle between two values of its
type with a chance of about 25000 * 2^-45 * 2^9 < 10^-6: they are compared as they
are."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import attn as oa
from oracle import serve as osv
from test_gpu_kv import DT, I32, new_cache, tables, values
from test_gpu_norm import N

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype,layout,D,rotary", [("f32", "half", 128, 128), ("f32", "interleaved", 64, 32),
                                                   ("bf16", "half", 256, 64), ("f32", "half", 80, 24)])
@pytest.mark.parametrize("size", [1.0, 1e-20, 1e18, 1e25, 1e36])
def test_keys_are_the_nearest_values(cache, dtype, layout, D, rotary, size):
    """Rows whose squares' sum passes binary32's range too: their norms are as others'."""
    new, total, heads = [20, 1, 28], [50, 1, 200], 2
    g = torch.Generator(device="cuda").manual_seed(D + rotary)
    pages, table, start = tables(new, total, 16)
    rows = int(start[-1])
    k = (torch.randn((rows, heads, D), generator=g, device="cuda") * size).to(DT[dtype])
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    f, _ = sv.sv_rope_frequencies(rotary, device="cuda")
    c = new_cache(cache, pages, 16, heads, D)
    sv.sv_kv_append_normed(k, k, c["k_cache"], c["v_cache"], I32(table), I32(start), I32(total), k_weight=w, freq=f,
                           layout=layout, k_scale=c["k_scale"], v_scale=c["v_scale"])
    place = np.array([oa.place_of(start, total, b, i) for b in range(3) for i in range(new[b])])
    want = osv.norm_rope(N(k), N(w), 1e-6, place, N(f), layout)
    if cache == "bf16":
        want = torch.from_numpy(want.astype(np.float32)).bfloat16().double().numpy()
    else:
        code, e = oa.quantise(want)
        want = oa.e4m3_values()[code] * np.exp2(e)[..., None]
    at = [(table[b, p // 16], p % 16) for b, p in zip(np.repeat(np.arange(3), new), place)]
    got = values(c, "k")[[x[0] for x in at], [x[1] for x in at]]
    assert np.array_equal(got, want), (got != want).sum()
