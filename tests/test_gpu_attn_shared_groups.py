"""sv_paged_attention_shared where a group's requests are not all in the batch:
such a group shares nothing, and no scratch is read that no part was written to.
Tolerances as in test_gpu_attn_shared.py."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from test_gpu_attn_shared import batch, call, oracle
from test_gpu_attn_sinks import within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

BAD = [  # group starts of a batch of three, and the groups that stand
    ([-3, 2], []), ([0, 9], []), ([2, 1], []), ([-1, 0, 2, 7], [1]), ([0, 2, 4], [0]), ([3, 5], []),
    ([-2 ** 31, 2 ** 31 - 1], []),
]


@pytest.mark.parametrize("new,q_heads,D", [([2, 1, 3], 4, 64), ([9, 1, 3], 4, 128), ([50, 1, 3], 4, 64), ([2, 1, 3], 2, 256)])
@pytest.mark.parametrize("groups,stand", BAD)
def test_groups_outside_the_batch_share_nothing(groups, stand, new, q_heads, D):
    n = len(groups) - 1
    s = batch("bf16", new, [80, 39, 61], [0, 2], [20], 16, 1, q_heads, D)
    want = oracle(dict(s, groups=[x for g in stand for x in groups[g:g + 2]], shared=[20] * len(stand)), D ** -0.5)
    s["groups"], s["shared"] = groups, [20] * n
    rows = sum(new)
    size = sv.sv_paged_attention_shared_workspace_size(3, rows, n, q_heads, 1, D, 0, 0, s["table"].shape[1] * 16,
                                                       s["table"].shape[1] * 16)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaNs
    o = call(s, workspace=ws)
    within(o, want, D, np.arange(rows))
