"""sv_paged_attention_shared with so many rows that a wave joins the parts of four
or eight of a token's heads (from 8193 and 32769 rows of heads on): head numbers
that these do not divide, and requests of several tiles of rows.  Tolerances as in
test_gpu_attn_shared.py."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from test_gpu_attn_shared import batch, call, hints, oracle
from test_gpu_attn_sinks import within
from test_gpu_kv import I32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]

SHAPES = [  # new tokens (of a request, of some others), requests, groups, kv heads, q heads, D
    ((2, 9), 296, [0, 100, 290], 2, 14, 64),    # 16 rows a tile, four heads a wave; requests of 63 rows
    ((5, 20), 220, [3, 220], 5, 30, 64),        # 32 rows a tile, eight heads a wave; requests of 120 rows
    ((5, 50), 120, [0, 60, 120], 1, 14, 128),   # 128 rows a tile; requests of 700 rows
    ((3, 30), 450, [0, 448], 2, 6, 256),        # four channels a lane
    ((9, 40), 520, [0, 5, 500], 1, 7, 80),
]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_many_rows_are_joined(cache, shape):
    (few, many), B, groups, heads, q_heads, D = SHAPES[shape]
    rng = np.random.default_rng(shape)
    new = [many if b % 97 == 50 else few for b in range(B)]
    shared = [40 - 9 * g for g in range(len(groups) - 1)]
    total = [int(rng.integers(30, 110)) for _ in range(B)]
    s = batch(cache, new, total, groups, shared, 16, heads, q_heads, D, seed=shape)
    rows = int(s["start"][-1])
    assert rows * q_heads > (32768 if shape == 1 else 8192)
    o = call(s, max_q_len=few)
    want = oracle(s, D ** -0.5)
    within(o, want, D, np.arange(rows))
    within(call(s, **hints(s)), want, D, np.arange(rows))
    again = call(s, max_q_len=few)
    assert torch.equal(o["out"], again["out"]) and torch.equal(o["lse"], again["lse"])
    # strided outputs, without lse
    wide = torch.full((rows, q_heads + 1, D), 9.0, device="cuda", dtype=torch.bfloat16)
    c = s["c"]
    sv.sv_paged_attention_shared(s["q"], c["k_cache"], c["v_cache"], I32(s["table"]), I32(s["start"]), I32(s["total"]),
                                 I32(s["groups"]), I32(s["shared"]), k_scale=c["k_scale"], v_scale=c["v_scale"],
                                 max_q_len=few, out=dict(out=wide[:, 1:]))
    assert torch.equal(wide[:, 1:], o["out"]) and (wide[:, 0] == 9.0).all()
