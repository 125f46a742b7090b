"""Windows, hints and sizes of sv_paged_attention that do not fit the C call's 32
bits: what is beyond every context counts as that, and nothing wraps around."""
import sys

import pytest
import torch

import draft_token_verification_spec_amd as sv
from test_gpu_attn import call, fill
from test_gpu_kv import I32, new_cache, tables

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("wide", [(1 << 31) - 1, 1 << 31, (1 << 32) + 1, 1 << 40, sys.maxsize])
def test_attention_of_wide_windows_and_hints(wide, new):
    pages, table, start = tables([new], [700], 16)
    c = fill(new_cache("bf16", pages, 16, 2, 64), 1)
    q = torch.randn((new, 4, 64), device="cuda").bfloat16()
    want = call(q, c, table, start, [700], max_q_len=new, max_kv_len=(1 << 31) - 1)
    got = call(q, c, table, start, [700], max_q_len=wide, max_kv_len=wide, window=wide)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    for kw in (dict(window=-wide), dict(window=1 - wide * 2), dict(max_q_len=-wide), dict(max_kv_len=-wide)):
        with pytest.raises(RuntimeError, match="invalid argument"):
            call(q, c, table, start, [700], **kw)


def test_more_rows_than_a_call_has():
    c = new_cache("bf16", 2, 16, 1, 16)
    k, v, table = c["k_cache"], c["v_cache"], I32([[0, 1]])
    one = torch.ones((1, 1, 16), device="cuda", dtype=torch.bfloat16)
    for T in ((1 << 23) + 1, (1 << 32) + 3):
        many = one.expand(T, 1, 16)
        with pytest.raises(ValueError, match="rows"):
            sv.sv_kv_append(many, many, k, v, table, I32([0, 3]), I32([3]))
        with pytest.raises(ValueError, match="rows"):
            sv.sv_paged_attention(many, k, v, table, I32([0, 3]), I32([3]), out=dict(out=many))
        with pytest.raises(ValueError, match="rows"):
            sv.sv_rope(many, torch.zeros(1, dtype=torch.int64, device="cuda").expand(T), None, out=many)
        with pytest.raises(ValueError, match="rows"):
            sv.sv_kv_gather(k, v, table, I32([0, 3]), T)
    assert (k == 3.0).all() and (v == 3.0).all()
