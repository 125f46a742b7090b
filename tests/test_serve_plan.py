"""How the attention variants of a served batch divide their work, as far as their
workspaces' sizes tell (no GPU)."""
import os

import pytest

import draft_token_verification_spec_amd as sv

pytestmark = pytest.mark.skipif(not os.path.exists(sv.lib_path()), reason="libspecverify.so not built")


@pytest.mark.parametrize("batch,new", [(64, 1), (64, 5), (256, 1), (256, 5)])
def test_long_windows_divide_contexts(batch, new):
    """Contexts are even only as far as their windows are short: behind a long one, what a row sees differs from request
    to request as it does without, and a long context among short ones is divided as there."""
    size, plain = sv.sv_paged_attention_sinks_workspace_size, sv.sv_paged_attention_workspace_size
    a = (batch, batch * new, 32, 8, 128, new)
    for window in (20000, 50000, 100000, 131000):
        part = batch * new * 32 * (128 * 4 + 8)
        want = min(8, -(-window // 16384))
        assert size(*a, 131072, window, 4) >= 256 + want * part, window
        assert size(*a, 131072, window, 4) <= plain(*a, 131072) + part, window
    assert size(*a, 131072, 2048, 4) == 256
