"""Refusals of the calls with several axes, of MXFP8 caches, of reading a cache back and of
attention over wide caches, without a GPU: every call here ends in the argument checks (stand-in
device addresses are only compared) or asks for no work."""

import ctypes
import os

import pytest

import layerwise_qk_norm_qknorm_amd as qk
from layerwise_qk_norm_qknorm_amd.binding import Axes
from test_operators_abi_cpu import (BF16, F32, FP8, INVALID, OK, UNSUPPORTED, at, batch, cache, grad, message, operand,
                                    rope)

pytestmark = pytest.mark.skipif(not os.path.exists(qk.library_path()),
                                reason="libqknorm.so not built (run __graft_entry__.build())")
MXFP8 = 3
THREE = bytes([0] * 16 + [1] * 24 + [2] * 24)


def axes(n=3, axis=THREE, ld=1000):
    return Axes(n, axis, ld)


def ref(x):
    return ctypes.byref(x) if x is not None else None


def call_rope(q=None, k=None, T=5, dtype=BF16, r=None, a=None):
    return qk.load_library().qknorm_headwise_rope_axes(ref(q or operand(0)), ref(k or operand(5)), T, dtype, 1e-6, 128,
                                                       0, ref(r or rope()), ref(a or axes()), None)


def call_grad(q=None, k=None, T=5, dtype=BF16, r=None, a=None, ws=at(50), nb=1 << 30):
    return qk.load_library().qknorm_headwise_rope_axes_backward(ref(q or grad(0)), ref(k or grad(8)), T, dtype, 1e-6,
                                                                128, 0, ref(r or rope()), ref(a or axes()), ws, nb,
                                                                None)


def eight(**kw):
    f = dict(format=MXFP8, page_stride=4 * 16 * 128, head_stride=16 * 128, token_stride=128)
    f.update(kw)
    return cache(**f)


def call_append(q=None, T=5, dtype=BF16, r=None, a=None, c=None, slots=at(45)):
    return qk.load_library().qknorm_paged_append_axes(ref(q or operand(0)), ref(operand(5, y=None)),
                                                      ref(operand(10, y=None)), T, dtype, 1e-6, 128, 0,
                                                      ref(r or rope()), ref(a or axes()), ref(c or eight()), slots,
                                                      None)


def call_gather(c=None, d=128, slots=at(45), T=5, dtype=BF16, k=at(60), ld_k=512, v=at(61), ld_v=512):
    return qk.load_library().qknorm_paged_gather(ref(c or eight()), d, slots, T, dtype, k, ld_k, v, ld_v, None)


def call_attend(q=None, T=6, dtype=BF16, c=None, d=128, b=None, scale=0.1, causal=1, window=0, ws=at(50), nb=1 << 34):
    return qk.load_library().qknorm_paged_attend_wide(ref(q or operand(0, h=1024)), T, dtype, ref(c or eight()), d,
                                                      ref(b or batch()), scale, causal, window, ws, nb, None)


@pytest.mark.parametrize("kw,text", [
    (dict(a=axes(n=0)), "n_axes"),
    (dict(a=axes(n=5)), "n_axes"),
    (dict(a=axes(axis=None)), "axis is required"),
    (dict(a=axes(n=2)), "axis 2 of angle 40"),
    (dict(a=axes(ld=-1)), "ld_positions"),
    (dict(a=axes(ld=1 << 62)), "ld_positions"),
    (dict(T=-1), "T = -1"),
    (dict(r=rope(positions=None)), "positions"),
    (dict(r=rope(rot_dim=130)), "rot_dim"),
    (dict(q=None, dtype=7), "unknown dtype"),
])
@pytest.mark.parametrize("call", [call_rope, call_grad, call_append])
def test_axes_refusals(call, kw, text):
    assert call(**kw) == INVALID, message()
    assert text in message()


def test_outputs_may_not_overlap_the_last_axis():
    ld = 1 << 20
    second = at(21) + 2 * ld * 8                     # where the third axis' positions lie
    assert call_rope(q=operand(0, y=second), a=axes(ld=ld)) == INVALID and "positions" in message()
    assert call_grad(q=grad(0, dx=second), a=axes(ld=ld)) == INVALID and "overlaps an input" in message()
    assert call_append(q=operand(0, y=second), a=axes(ld=ld)) == INVALID and "positions" in message()


def test_axes_without_rotation_are_not_looked_at():
    none = dict(x=None, y=None, gamma=None)
    assert call_rope(T=0, q=operand(0, **none), k=operand(5, **none), r=rope(rot_dim=0), a=axes(n=9)) == OK
    assert call_rope(T=0, q=operand(0, **none), k=operand(5, **none), a=axes(n=9)) == INVALID


@pytest.mark.parametrize("kw,code,text", [
    (dict(dtype=FP8), UNSUPPORTED, "FP8"),
    (dict(c=eight(format=4)), INVALID, "format"),
    (dict(c=eight(format=2)), INVALID, "format"),
    (dict(c=eight(page_size=8)), INVALID, "MXFP8 pages hold at least 16"),
    (dict(c=eight(token_stride=120)), INVALID, "strides"),
    (dict(c=eight(token_stride=136)), INVALID, "MXFP8 token strides"),
    (dict(c=eight(head_stride=16 * 128 - 128)), INVALID, "overlap"),
    (dict(c=eight(page_stride=4 * 16 * 128 + 8)), INVALID, "16 bytes"),
    (dict(c=eight(k_scales=None)), INVALID, "cache pointers"),
    (dict(c=eight(v=at(31) + 8)), INVALID, "16-byte"),
    (dict(c=eight(scale_head_stride=48)), INVALID, "overlap"),
    (dict(c=eight(v=at(30))), INVALID, "overlaps"),
    (dict(c=eight(v_scales=at(32))), INVALID, "overlaps"),
    (dict(q=operand(0, y=at(33))), INVALID, "overlaps"),
    (dict(slots=None), INVALID, "slots"),
])
def test_append_refusals(kw, code, text):
    assert call_append(**kw) == code, message()
    assert text in message()


@pytest.mark.parametrize("kw,code,text", [
    (dict(dtype=FP8), UNSUPPORTED, "FP8"),
    (dict(dtype=9), INVALID, "unknown dtype"),
    (dict(T=-1), INVALID, "T = -1"),
    (dict(d=0), INVALID, "head_dim"),
    (dict(d=2048), UNSUPPORTED, "head_dim"),
    (dict(c=eight(format=2)), INVALID, "format"),
    (dict(c=eight(k=None)), INVALID, "cache pointers"),
    (dict(c=eight(n_pages=0)), INVALID, "pages"),
    (dict(k=None, v=None), INVALID, "k_rows or v_rows"),
    (dict(ld_k=511), INVALID, "k_rows row stride"),
    (dict(v=at(61) + 1), INVALID, "aligned"),
    (dict(slots=None), INVALID, "slots"),
    (dict(slots=at(45) + 4), INVALID, "slots"),
    (dict(v=at(60)), INVALID, "k_rows overlaps v_rows"),
    (dict(k=at(30)), INVALID, "overlap the cache"),
    (dict(v=at(33)), INVALID, "overlap the cache"),
    (dict(k=at(45)), INVALID, "overlap the cache or slots"),
    (dict(d=80, c=eight(heads=4)), INVALID, "multiple of 32"),
    (dict(T=1 << 60), INVALID, "address range"),
])
def test_gather_refusals(kw, code, text):
    assert call_gather(**kw) == code, message()
    assert text in message()


def rows(**kw):
    return cache(four=False, **kw)


@pytest.mark.parametrize("kw,code,text", [
    (dict(T=-1), INVALID, "T = -1"),
    (dict(dtype=F32), UNSUPPORTED, "bf16"),
    (dict(d=96), UNSUPPORTED, "head_dim"),
    (dict(c=cache()), UNSUPPORTED, "rows or MXFP8"),
    (dict(c=eight(format=2)), INVALID, "format"),
    (dict(scale=0.0), INVALID, "scale"),
    (dict(window=-1), INVALID, "window"),
    (dict(c=eight(heads=3)), INVALID, "key heads"),
    (dict(c=rows(page_size=8)), UNSUPPORTED, "16 tokens"),
    (dict(c=rows(k=at(30) + 8)), INVALID, "16 bytes"),
    (dict(c=rows(token_stride=132)), INVALID, "16 bytes"),
    (dict(c=rows(page_stride=4 * 16 * 128 + 4)), INVALID, "16 bytes"),
    (dict(c=rows(token_stride=1 << 28, head_stride=128)), UNSUPPORTED, "token_stride"),
    (dict(q=operand(0, h=1024, x=at(0) + 8)), INVALID, "16-byte"),
    (dict(q=operand(0, h=1024, y=at(30))), INVALID, "overlaps"),
    (dict(q=operand(0, h=1024, y=at(33))), INVALID, "overlaps"),
    (dict(b=batch(B=-1)), INVALID, "batch"),
    (dict(b=batch(cu_q=None)), INVALID, "without cu_q"),
    (dict(b=batch(block_table=None)), INVALID, "block_table"),
    (dict(b=batch(B=1 << 21)), UNSUPPORTED, "limits"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), ws=None), INVALID, "workspace"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), nb=64), INVALID, "workspace"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), ws=at(30)), INVALID, "overlaps"),
])
def test_attend_refusals(kw, code, text):
    assert call_attend(**kw) == code, message()
    assert text in message()


def test_rows_of_one_allocation_overlap_what_lies_in_them():
    """bf16 strides count elements: a V that begins inside K's pages is seen, and so is an output
    behind the middle of the cache."""
    c = rows()
    behind = at(30) + 2 * 9 * 4 * 16 * 128            # the last page, in bytes
    assert call_attend(c=c, q=operand(0, h=1024, y=behind)) == INVALID and "overlaps" in message()
    assert call_gather(c=c, k=behind) == INVALID and "overlap" in message()


def test_mxfp4_attention_still_names_its_format():
    lib = qk.load_library()
    for c in (eight(), rows()):
        assert lib.qknorm_paged_attend(ref(operand(0, h=1024)), 6, BF16, ref(c), 128, ref(batch()), 0.1, 1, 0, at(50),
                                       1 << 34, None) == UNSUPPORTED and "MXFP4" in message()


def test_calls_for_no_work():
    none = dict(x=None, y=None, gamma=None)
    empty = dict(k=None, v=None, k_scales=None, v_scales=None)
    assert call_rope(T=0, q=operand(0, **none), k=operand(5, **none), r=rope(cos_sin=None, positions=None)) == OK
    assert call_grad(T=0, ws=None, nb=0) == OK
    assert call_append(T=0, slots=None, c=eight(**empty)) == OK
    assert call_gather(T=0, slots=None, k=None, v=None, c=eight(**empty)) == OK
    assert call_attend(T=0, b=batch(B=0), ws=None, nb=0, c=rows(**empty)) == OK


def test_workspace_sizes():
    lib = qk.load_library()
    for rows_q in (1, 5, 40, 600):
        sizes = [lib.qknorm_paged_attend_wide_workspace(rows_q, 40, 8, 128, 1, rows_q, n) for n in range(64, 1 << 16, 777)]
        assert sizes == sorted(sizes)           # never less for a longer cache
        assert sizes[-1] > 0
    assert lib.qknorm_paged_attend_wide_workspace(1, 40, 8, 128, 1, 1, 64) == 0
    assert lib.qknorm_paged_attend_wide_workspace(1, 40, 7, 128, 1, 1, 4096) == 0


def test_axes_helper():
    assert qk.rope_axes((16, 24, 24)) == THREE
    assert qk.rope_axes((1, 3, 2), spread=True) == bytes([0, 1, 2, 1, 2, 1])
    assert qk.rope_axes((4,)) == bytes(4)
    for bad in ((), (1, -1), (1, 1, 1, 1, 1)):
        with pytest.raises(ValueError):
            qk.rope_axes(bad)
