"""Sizes that the attention calls refuse need no workspace, without a GPU."""

import os

import pytest

import layerwise_qk_norm_qknorm_amd as qk
from test_operators_abi_cpu import UNSUPPORTED, at, batch, message, operand
from test_wide_abi_cpu import call_attend

pytestmark = pytest.mark.skipif(not os.path.exists(qk.library_path()),
                                reason="libqknorm.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("name", ["qknorm_paged_attend_workspace", "qknorm_paged_attend_wide_workspace"])
@pytest.mark.parametrize("group", [1, 5, 8])
def test_rows_beyond_the_limit_need_no_workspace(name, group):
    """At most 2^28 rows of a key head's query heads; one sequence of 2^20 tokens is split below that."""
    size = getattr(qk.load_library(), name)
    most = (1 << 28) // group
    assert size(most, group, 1, 128, 1, 1, 1 << 20) > 0
    for T in (most + 1, 1 << 31, 1 << 44, 1 << 62):
        assert size(T, group, 1, 128, 1, 1, 1 << 20) == 0


def test_such_rows_are_refused_before_their_workspace():
    T = (1 << 28) // 2 + 1       # 8 query heads on 4 key heads
    b = batch(table_pages=1 << 16, ld_table=1 << 16, max_len=1 << 20)
    assert call_attend(q=operand(0, h=1024), T=T, b=b, ws=at(600), nb=64) == UNSUPPORTED, message()
    assert "too many" in message()
