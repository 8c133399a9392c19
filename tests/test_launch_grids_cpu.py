"""The grids that the operators around headwise QK-Norm launch, without a GPU."""

import os

import pytest

import layerwise_qk_norm_qknorm_amd as qk
from launch_grids import grids

pytestmark = pytest.mark.skipif(not os.path.exists(qk.library_path()),
                                reason="libqknorm.so not built (run __graft_entry__.build())")


def attend(T, B, max_q, max_len=512, heads_q=40, heads_k=8, d=128, ps=16):
    """A call of T query rows in B sequences."""
    far = 1 << 52       # the rows lie behind every other stand-in buffer
    row = heads_k * ps * d // 2
    return ["attend", dict(
        T=T, d=d,
        q=["operand", dict(i=0, h=heads_q * d, x=far, y=2 * far, ld_x=heads_q * d, ld_y=heads_q * d)],
        c=["cache", dict(heads=heads_k, page_size=ps, token_stride=d // 2, head_stride=ps * d // 2, page_stride=row,
                         scale_head_stride=ps * d // 32, scale_page_stride=row // 16)],
        b=["batch", dict(B=B, max_q=max_q, max_len=max_len, table_pages=max_len // ps, ld_table=max_len // ps)])]


def test_attention_without_a_bound_on_the_rows(tmp_path):
    """Ragged batches with max_q left at the row count, which is what a call without the hint
    passes: they launch, with no more blocks than a few times those that find rows (or 2^17)."""
    calls = [(120000, 256), (60000, 512), (8192, 4096), (16609, 512), (30098, 256), (8192, 1), (1 << 20, 1 << 15)]
    for (T, B), (rc, message, launches) in zip(calls, grids([attend(T, B, T) for T, B in calls], tmp_path)):
        assert rc == 0, (T, B, message)
        assert len(launches) == 1
        blocks, _, threads = launches[0]
        full = 8 * (T * 5 / 64 + B)         # row tiles that can hold a row, with those cut at a sequence's end
        assert blocks <= max(5 * full, 2 ** 17, 64 * 8 * B), (T, B, blocks)
        assert blocks * threads < 2 ** 32


def test_attention_grids_that_fit_stay_as_the_bound_asks(tmp_path):
    """Up to 2^17 blocks every sequence gets those of max_q rows."""
    calls = [(1024, 64, 1024), (8192, 1, 8192), (8192, 64, 300), (2303, 255, 200)]
    for (T, B, q), (rc, message, launches) in zip(calls, grids([attend(*c) for c in calls], tmp_path)):
        assert rc == 0, message
        assert launches[0][0] == B * 8 * -(-q * 5 // 64), (T, B, q)
