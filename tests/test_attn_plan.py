"""How sv_paged_attention divides its work, as far as its workspace's size tells
(no GPU)."""
import os

import pytest

import draft_token_verification_spec_amd as sv

pytestmark = pytest.mark.skipif(not os.path.exists(sv.lib_path()), reason="libspecverify.so not built")

INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("batch,rows,q_heads,heads,D,max_q", [
    (8, 8, 32, 8, 128, 1), (1, 1, 32, 8, 128, 1), (1, 5, 8, 8, 64, 5), (4, 80, 32, 4, 128, 20), (300, 300, 32, 8, 128, 1),
])
def test_longest_hint_is_the_largest_cache(batch, rows, q_heads, heads, D, max_q):
    """A hint beyond what a page table can hold says no more than that much does."""
    sizes = [sv.sv_paged_attention_workspace_size(batch, rows, q_heads, heads, D, max_q, kv)
             for kv in (sv.SV_ATTN_MAX_TOKENS, sv.SV_ATTN_MAX_TOKENS + 1, INT_MAX - 300, INT_MAX - 16000, INT_MAX)]
    assert len(set(sizes)) == 1, sizes
