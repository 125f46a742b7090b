"""How sv_paged_attention divides its work, as far as its workspace's size tells
(no GPU)."""
import math
import os
import random
import sys

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


def test_scratch_is_bounded():
    """Parts of divided contexts take at most 2^29 bytes, however many rows, long contexts or loose hints a call has."""
    size = sv.sv_paged_attention_workspace_size
    rng = random.Random(1)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    cases = [(4096, 20480, 32, 8, 128, 5, 131072), (4096, 20480, 32, 8, 128, 0, 131072), (1 << 18, 1 << 20, 128, 8, 256, 1, 1 << 30),
             (1 << 18, 1 << 21, 1023, 1, 16, 0, INT_MAX), (1, 1, 1024, 1024, 256, 1, INT_MAX)]
    for _ in range(20000):
        heads = log(1, 64)
        q_heads = heads * log(1, 1024 // heads)
        batch, rows = log(1, 1 << 18), log(1, min(1 << 23, INT_MAX // q_heads))
        cases.append((batch, rows, q_heads, heads, 16 * log(1, 16), rng.choice([0, 1, 5, log(1, rows)]), log(1, INT_MAX)))
    for case in cases:
        assert 256 <= size(*case) <= (1 << 29) + 1024, case
    # and a context among few enough is still divided
    assert size(256, 1280, 32, 8, 128, 5, 131072) > 8 * 1280 * 32 * 128 * 4


def test_hints_beyond_32_bits():
    """Python's integers have no end; a hint of any size says what the largest says."""
    size = sv.sv_paged_attention_workspace_size
    want = size(8, 8, 32, 8, 128, 1, INT_MAX)
    assert want > 256
    for kv in (1 << 31, (1 << 32) + 5, 1 << 40, sys.maxsize):
        assert size(8, 8, 32, 8, 128, 1, kv) == want
        assert size(8, 8, 32, 8, 128, kv, INT_MAX) == size(8, 8, 32, 8, 128, 8, INT_MAX)
    assert size(8, 8, 32, 8, 128, 1, -1) == size(8, 8, 32, 8, 128, 1, 5 - (1 << 32)) == 0


@pytest.mark.parametrize("scale,status", [(2.3e38, 0), (2.36e38, -1), (3.4e38, -1), (1e-45, 0), (0.0, -1)])
def test_scale_in_base_two_is_finite(scale, status):
    """Scores are formed in base 2: a scale that is infinite there is refused (no row: what is let pass does nothing)."""
    from test_attn_abi import attention

    assert attention(T=0, scale=scale) == status
