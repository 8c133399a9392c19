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


def rope(T, heads_q, heads_k, d, dtype=1, rot=None, inter=0, **kw):
    """A call of the rotation: packed rows, Q then K."""
    far, ld = 1 << 52, (heads_q + heads_k) * d
    e = 4 if dtype == 0 else 2 if dtype == 1 else 1
    side = lambda i, h, at: ["operand", dict(i=i, h=h * d, x=far + at * e, y=2 * far + at * e, ld_x=ld, ld_y=ld)]
    rot = d if rot is None else rot
    return ["rope", dict(T=T, d=d, dtype=dtype, q=side(0, heads_q, 0), k=side(5, heads_k, heads_q * d),
                         r=["rope", dict(rot_dim=rot, ld=max(rot, 1), interleaved=inter)])]


def append(T, heads_q, heads_k, d, four=True, ps=16, dtype=1, rot=None, inter=0):
    far, ld = 1 << 52, (heads_q + 2 * heads_k) * d
    e = 4 if dtype == 0 else 2
    row = lambda i, h, at, y: ["operand", dict(i=i, h=h * d, x=far + at * e, y=y, ld_x=ld, ld_y=heads_q * d)]
    unit = d // 2 if four else d
    c = dict(four=four, heads=heads_k, page_size=ps, n_pages=4, token_stride=unit, head_stride=ps * unit,
             page_stride=heads_k * ps * unit)
    if four:
        c.update(scale_head_stride=ps * d // 32, scale_page_stride=heads_k * ps * d // 32)
    rot = d if rot is None else rot
    return ["append", dict(T=T, d=d, dtype=dtype, q=row(0, heads_q, 0, 2 * far), k=row(5, heads_k, heads_q * d, None),
                           v=row(10, heads_k, (heads_q + heads_k) * d, None),
                           r=["rope", dict(rot_dim=rot, ld=max(rot, 1), interleaved=inter)], c=["cache", c])]


def test_the_cap_on_blocks_holds_for_the_whole_grid(tmp_path):
    """Of both layouts (heads of 320 columns: 24 blocks' worth of waves in three blocks a token)."""
    calls = [rope(100, 40, 8, 320), rope(5000, 40, 8, 128), rope(100, 9, 3, 81, rot=80), rope(5000, 40, 8, 80),
             append(100, 40, 8, 320), append(5000, 10, 2, 128), append(100, 40, 8, 320, four=False),
             append(5000, 10, 2, 128, four=False)]
    free, capped = grids(calls, tmp_path), grids(calls, tmp_path, cap=7)
    for call, (rc, message, launches), (_, _, most) in zip(calls, capped, free):
        assert rc == 0, message
        assert max(x * y for x, y, _ in most) > 7, call
        assert max(x * y for x, y, _ in launches) <= 7, (call, launches)
    # never less than the blocks of one token
    rc, message, launches = grids([rope(100, 40, 8, 320)], tmp_path, cap=1)[0]
    assert rc == 0 and launches == [[1, 3, 512]], (message, launches)


SIZES = {"f32": 4, "bf16": 2, "fp8": 1}
CODES = {"f32": 0, "bf16": 1, "fp8": 2}


def _waves(dtype, heads, d, layout, slots):
    """Slots of each side, and the waves that a token's take."""
    chunk = 16 // SIZES[dtype]
    lanes = 1
    while lanes < (d // chunk if layout == "whole" else d // (2 * chunk)):
        lanes *= 2
    per_side = [-(-h * lanes // 64) for h in heads]
    if layout == "whole":
        return sum(-(-n // slots) for n in per_side), per_side
    return -(-sum(per_side) // slots), per_side


def _expected(T, dtype, heads, d, layout, slots):
    waves, _ = _waves(dtype, heads, d, layout, slots)
    if layout == "whole":       # four waves to a block, tokens one after the other
        return [-(-T * waves // 4), 1, 256]
    tokens = 1 if waves >= 4 else 4 // waves
    assert waves <= 8
    return [-(-T // tokens), 1, 64 * waves * tokens]


def test_the_variants_are_the_ones_that_the_gpu_tests_mean(tmp_path):
    """operator_variants.py names the layout and slots that each of its calls takes."""
    from operator_variants import APPEND, ROPE
    calls, want = [], []
    for (dtype, T, nq, nk, d, rot, inter, _, _), (layout, slots) in ROPE:
        calls.append(rope(T, nq, nk, d, dtype=CODES[dtype], rot=rot, inter=int(inter)))
        want.append([_expected(T, dtype, (nq, nk), d, layout, slots)])
    for kw, (layout, slots) in APPEND:
        T, dtype, nq, nk, d = (kw[n] for n in ("T", "dtype", "nq", "nk", "d"))
        for four in (True, False):
            calls.append(append(T, nq, nk, d, four=four, dtype=CODES[dtype], rot=kw["rot"], inter=int(kw["inter"])))
            if four and layout == "whole" and slots > 1:    # Q in a launch of its own
                want.append([_expected(T, dtype, (nq,), d, layout, slots),
                             _expected(T, dtype, (nk, nk), d, layout, slots)])
            else:
                want.append([_expected(T, dtype, (nq, nk, nk), d, layout, slots)])
    for call, launches, (rc, message, got) in zip(calls, want, grids(calls, tmp_path)):
        assert rc == 0, message
        assert got == launches, (call, got, launches)
