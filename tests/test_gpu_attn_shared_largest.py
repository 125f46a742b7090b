"""sv_paged_attention_shared with 2^29 rows of heads, whose parts are joined by more
threads than one dimension of a grid can hold."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import serve as osv
from test_gpu_attn import fill
from test_gpu_attn_sinks import N
from test_gpu_kv import I32, new_cache, values

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


def test_joins_beyond_a_grid_of_32_bits():
    """All rows have the same queries, and, but for the first 16, see the same 16 tokens (the page table holds no more): 8
    shared ones and 8 of their own."""
    T, heads, D, few = 1 << 19, 1024, 16, 40
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GiB")
    c = fill(new_cache("bf16", 1, 16, heads, D), 1)
    q = torch.randn((1, heads, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    o = sv.sv_paged_attention_shared(q.expand(T, heads, D), c["k_cache"], c["v_cache"], I32([[0]]), I32([0, T]), I32([T]),
                                     I32([0, 1]), I32([8]))["out"]
    cache = dict(k=values(c, "k"), v=values(c, "v"), table=np.array([[0]]))
    want = osv.attention(N(q.expand(few, heads, D)), cache, [0, few], [few], D ** -0.5)
    e = (D + 4) * 2.0 ** -24 * want["size"] + 2.0 ** -21  # (as in test_gpu_attn.py)
    tol = (2 * e[..., None] + 2 * 2.0 ** -8) * want["spread"] + np.abs(want["out"]) * 2.0 ** -8
    assert (np.abs(N(o[:few]) - want["out"]) <= tol).all()
    last = o[T - 1]
    assert all((x == last).all() for x in o[16:].split(1 << 16))
