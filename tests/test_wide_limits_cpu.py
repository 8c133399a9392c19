"""Limits of a launch that the calls over wide caches are held to, without a GPU: every call here
ends in the argument checks."""

import os

import pytest

import layerwise_qk_norm_qknorm_amd as qk
from test_operators_abi_cpu import UNSUPPORTED, at, batch, message, operand
from test_wide_abi_cpu import call_attend, eight

pytestmark = pytest.mark.skipif(not os.path.exists(qk.library_path()),
                                reason="libqknorm.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("max_q,heads,group", [
    (200, 64, 1),      # blocks of 512 threads: 2^23 of them are one more than a launch's 2^32 - 1 threads hold
    (64, 128, 1),      # of 256: 2^24
    (16, 128, 1),
    (100, 64, 2),
])
def test_launches_of_more_threads_than_there_are(max_q, heads, group):
    """One block per 256 (128, 16) rows of each of 2^17 sequences and key heads."""
    c = eight(heads=heads, page_stride=heads * 16 * 128, scale_page_stride=heads * 16 * 4)
    width = heads * group * 128
    q = operand(0, h=width, ld_x=width, ld_y=width)
    b = batch(B=1 << 17, max_q=max_q, table_pages=1, ld_table=1, max_len=16)
    assert call_attend(q=q, T=1 << 18, c=c, b=b, ws=at(600), nb=1 << 50) == UNSUPPORTED, message()
    assert "exceeds the grid" in message()
