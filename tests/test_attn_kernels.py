"""Which attention kernels the library holds: none that no call launches (no GPU)."""
import os
import re

import pytest

import draft_token_verification_spec_amd as sv

pytestmark = pytest.mark.skipif(not os.path.exists(sv.lib_path()), reason="libspecverify.so not built")


def test_splits_are_joined_by_themselves_for_whole_contexts_only():
    """Parts of the shared and the own tokens (kShared, kOwn: 2 and 3) are joined by kernels of their own."""
    with open(sv.lib_path(), "rb") as f:
        joins = set(re.findall(rb"11join_kernelILi(\d+)ELNS0_4PartE(\d)E", f.read()))
    assert joins == {(tile, part) for tile in (b"16", b"32", b"128") for part in (b"0", b"1")}
