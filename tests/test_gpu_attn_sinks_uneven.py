"""sv_paged_attention_sinks for batches whose requests and heads fill the card:
their contexts are not divided by a short window and are by a long one.  Contexts
of all lengths, also shorter than the window.  Tolerances as in
test_gpu_attn_sinks.py."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from test_gpu_attn import fill
from test_gpu_attn_sinks import call, oracle, within
from test_gpu_kv import new_cache, tables

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,window,sinks,divided", [(1, 500, 4, False), (3, 300, 70, False), (1, 18000, 4, True),
                                                      (3, 18000, 40, True)])
def test_contexts_of_all_lengths(cache, new, window, sinks, divided):
    B, heads, D = 64, 8, 64
    total = [5 + 17 * b % 900 for b in range(B)]
    total[1], total[7], total[40] = 20100 if divided else 4000, 0, 2500
    pages, table, start = tables([new] * B, total, 16, seed=new)
    c = fill(new_cache(cache, pages, 16, heads, D), new)
    q = torch.randn((B * new, heads, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    size = sv.sv_paged_attention_sinks_workspace_size(B, B * new, heads, heads, D, new, max(total), window, sinks)
    assert (size > 256) == divided
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaNs
    o = call(q, c, table, start, total, window=window, sinks=sinks, max_q_len=new, max_kv_len=max(total), workspace=ws)
    within(o, oracle(q, c, table, start, total, D ** -0.5, window, sinks), D, np.arange(B * new))
