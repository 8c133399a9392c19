"""Refusals of the operators around headwise QK-Norm, without a GPU: every
call here ends in the argument checks (stand-in device addresses are only
compared, never dereferenced) or asks for no work."""

import ctypes
import os

import pytest

import layerwise_qk_norm_qknorm_amd as qk
from layerwise_qk_norm_qknorm_amd.binding import Batch, Cache, GradOperand, Operand, Rope

pytestmark = pytest.mark.skipif(not os.path.exists(qk.library_path()),
                                reason="libqknorm.so not built (run __graft_entry__.build())")

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16, FP8 = 0, 1, 2
G = 1 << 40     # far apart stand-in buffers


def at(i):
    return (i + 1) * G


def rope(**kw):
    f = dict(cos_sin=at(20), ld=128, n_positions=100, positions=at(21), rot_dim=128, interleaved=0)
    f.update(kw)
    return Rope(*[f[n] for n, _ in Rope._fields_])


def operand(i, h=512, **kw):
    f = dict(x=at(i), ld_x=4096, y=at(i + 1), ld_y=4096, gamma=at(i + 2), h=h)
    f.update(kw)
    return Operand(*[f[n] for n, _ in Operand._fields_])


def grad(i, h=512, **kw):
    f = dict(x=at(i), ld_x=4096, dy=at(i + 1), ld_dy=4096, dx=at(i + 2), ld_dx=4096, gamma=at(i + 3),
             dgamma=at(i + 4), h=h)
    f.update(kw)
    return GradOperand(*[f[n] for n, _ in GradOperand._fields_])


def cache(four=True, **kw):
    f = dict(format=int(four), k=at(30), v=at(31), k_scales=at(32), v_scales=at(33), page_stride=4 * 16 * 64,
             head_stride=16 * 64, token_stride=64, scale_page_stride=4 * 64, scale_head_stride=64, n_pages=10,
             page_size=16, heads=4)
    if not four:
        f.update(page_stride=4 * 16 * 128, head_stride=16 * 128, token_stride=128)
    f.update(kw)
    return Cache(*[f[n] for n, _ in Cache._fields_])


def batch(**kw):
    f = dict(block_table=at(40), ld_table=8, table_pages=8, seq_lens=at(41), cu_q=at(42), B=3, max_q=4, max_len=100)
    f.update(kw)
    return Batch(*[f[n] for n, _ in Batch._fields_])


def message():
    return qk.load_library().qknorm_last_error().decode()


def call_rope(q=None, k=None, T=5, dtype=BF16, eps=1e-6, d=128, gs=0, r=None):
    q, k = q or operand(0), k or operand(5)
    r = rope() if r is None else r
    return qk.load_library().qknorm_headwise_rope(ctypes.byref(q), ctypes.byref(k), T, dtype, eps, d, gs,
                                                  ctypes.byref(r) if r else None, None)


def call_grad(q=None, k=None, T=5, dtype=BF16, eps=1e-6, d=128, gs=0, r=None, ws=at(50), nb=1 << 30):
    q, k = q or grad(0), k or grad(8)
    r = rope() if r is None else r
    return qk.load_library().qknorm_headwise_rope_backward(ctypes.byref(q), ctypes.byref(k), T, dtype, eps, d, gs,
                                                           ctypes.byref(r) if r else None, ws, nb, None)


def call_append(q=None, k=None, v=None, T=5, dtype=BF16, eps=1e-6, d=128, gs=0, r=None, c=None, slots=at(45)):
    k, v = k or operand(5, y=None), v or operand(10, y=None)
    r, c = r or rope(), c or cache()
    return qk.load_library().qknorm_paged_append(ctypes.byref(q or operand(0)), ctypes.byref(k), ctypes.byref(v), T,
                                                 dtype, eps, d, gs, ctypes.byref(r), ctypes.byref(c), slots, None)


def call_attend(q=None, T=6, dtype=BF16, c=None, d=128, b=None, scale=0.1, causal=1, window=0, ws=at(50), nb=1 << 34):
    q = q or operand(0, h=1024)
    return qk.load_library().qknorm_paged_attend(ctypes.byref(q), T, dtype, ctypes.byref(c or cache()), d,
                                                 ctypes.byref(b or batch()), scale, causal, window, ws, nb, None)


COMMON = [
    (dict(T=-1), INVALID, "T = -1"),
    (dict(dtype=7), INVALID, "unknown dtype"),
    (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(d=0), INVALID, "head_dim"),
    (dict(d=96, r=rope(rot_dim=64)), INVALID, "multiple of head_dim"),
    (dict(gs=-1), INVALID, "gamma_head_stride"),
    (dict(r=rope(rot_dim=130)), INVALID, "rot_dim"),
    (dict(r=rope(rot_dim=-2)), INVALID, "rot_dim"),
    (dict(r=rope(rot_dim=7)), INVALID, "rot_dim"),
    (dict(r=rope(ld=127)), INVALID, "rope->ld"),
    (dict(r=rope(n_positions=0)), INVALID, "n_positions"),
    (dict(r=rope(cos_sin=None)), INVALID, "cos_sin"),
    (dict(r=rope(positions=None)), INVALID, "positions"),
    (dict(r=rope(positions=at(21) + 4)), INVALID, "aligned"),
    (dict(r=rope(cos_sin=at(20) + 2)), INVALID, "aligned"),
]


@pytest.mark.parametrize("kw,code,text", COMMON)
@pytest.mark.parametrize("call", [call_rope, call_grad, call_append])
def test_shared_refusals(call, kw, code, text):
    assert call(**kw) == code, message()
    assert text in message()


@pytest.mark.parametrize("kw,code,text", [
    (dict(d=2048, q=operand(0, h=2048), k=operand(5, h=2048), r=rope(rot_dim=0)), UNSUPPORTED, "head_dim"),
    (dict(q=operand(0, x=None)), INVALID, "q->x"),
    (dict(q=operand(0, y=None)), INVALID, "q->y"),
    (dict(q=operand(0, gamma=None)), INVALID, "gamma"),
    (dict(q=operand(0, ld_x=511)), INVALID, "stride"),
    (dict(q=operand(0, x=at(0) + 1)), INVALID, "aligned"),
    (dict(q=operand(0, gamma=at(2) + 1)), INVALID, "aligned"),
    (dict(q=operand(0, y=at(0) + 2)), INVALID, "overlaps"),                 # partly its own input
    (dict(q=operand(0, y=at(5))), INVALID, "overlaps"),                     # the other side's input
    (dict(q=operand(0, y=at(6))), INVALID, "overlaps"),                     # the other side's output
    (dict(q=operand(0, y=at(20))), INVALID, "overlaps"),                    # the table
    (dict(q=operand(0, y=at(21))), INVALID, "overlaps"),                    # positions
    (dict(q=operand(0, y=at(7))), INVALID, "overlaps"),                     # gamma
    (dict(T=1 << 55), INVALID, "address range"),
])
def test_forward_refusals(kw, code, text):
    assert call_rope(**kw) == code, message()
    assert text in message()


@pytest.mark.parametrize("kw,code,text", [
    (dict(dtype=FP8), UNSUPPORTED, "FP8"),
    (dict(gs=64), INVALID, "gamma_head_stride"),
    (dict(q=grad(0, dy=None)), INVALID, "q->dy"),
    (dict(q=grad(0, dx=None)), INVALID, "q->dx"),
    (dict(q=grad(0, gamma=None)), INVALID, "gamma"),
    (dict(q=grad(0, dgamma=at(4) + 2)), INVALID, "dgamma"),
    (dict(ws=None), INVALID, "workspace"),
    (dict(ws=at(50) + 8), INVALID, "workspace"),
    (dict(nb=16), INVALID, "workspace"),
    (dict(q=grad(0, dx=at(8))), INVALID, "overlap"),
    (dict(q=grad(0, dx=at(1) + 2)), INVALID, "overlap"),
    (dict(q=grad(0, dgamma=at(10))), INVALID, "overlap"),
    (dict(q=grad(0, dgamma=at(50))), INVALID, "overlap"),
    (dict(ws=at(20)), INVALID, "overlap"),
])
def test_backward_refusals(kw, code, text):
    assert call_grad(**kw) == code, message()
    assert text in message()


@pytest.mark.parametrize("kw,code,text", [
    (dict(dtype=FP8), UNSUPPORTED, "FP8"),
    (dict(c=cache(format=2)), INVALID, "format"),
    (dict(c=cache(heads=3)), INVALID, "heads * head_dim"),
    (dict(c=cache(n_pages=0)), INVALID, "pages"),
    (dict(c=cache(page_size=24)), INVALID, "power of two"),
    (dict(c=cache(page_size=8)), INVALID, "16 tokens"),
    (dict(c=cache(token_stride=128)), INVALID, "packed"),
    (dict(c=cache(head_stride=16 * 64 - 64)), INVALID, "overlap"),
    (dict(c=cache(page_stride=16 * 64)), INVALID, "overlap"),
    (dict(c=cache(scale_head_stride=48)), INVALID, "overlap"),
    (dict(c=cache(page_stride=4 * 16 * 64 + 8)), INVALID, "16 bytes"),
    (dict(c=cache(k=None)), INVALID, "cache pointers"),
    (dict(c=cache(k_scales=None)), INVALID, "cache pointers"),
    (dict(c=cache(k=at(30) + 4)), INVALID, "16-byte"),
    (dict(c=cache(n_pages=1 << 60)), INVALID, "cache"),
    (dict(c=cache(v=at(30))), INVALID, "overlaps"),
    (dict(c=cache(four=False, token_stride=127)), INVALID, "strides"),
    (dict(c=cache(four=False, k=at(30) + 1)), INVALID, "aligned"),
    (dict(d=80, c=cache(heads=4), k=operand(5, h=320, y=None), v=operand(10, h=320, y=None), q=operand(0, h=320),
          r=rope(rot_dim=0)), INVALID, "multiple of 32"),
    (dict(slots=None), INVALID, "slots"),
    (dict(slots=at(45) + 4), INVALID, "slots"),
    (dict(k=operand(5, y=at(5))), INVALID, "overlaps"),                     # k and v rows are never in place
    (dict(q=operand(0, y=at(30))), INVALID, "overlaps"),                    # the cache
    (dict(v=operand(10, y=None, h=256)), INVALID, "heads * head_dim"),
    (dict(v=operand(10, x=None, y=None)), INVALID, "v->x"),
])
def test_append_refusals(kw, code, text):
    assert call_append(**kw) == code, message()
    assert text in message()


@pytest.mark.parametrize("kw,code,text", [
    (dict(T=-1), INVALID, "T = -1"),
    (dict(dtype=9), INVALID, "unknown dtype"),
    (dict(dtype=F32), UNSUPPORTED, "bf16"),
    (dict(d=96), UNSUPPORTED, "head_dim"),
    (dict(d=0), INVALID, "head_dim"),
    (dict(c=cache(four=False)), UNSUPPORTED, "MXFP4"),
    (dict(scale=0.0), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(window=-1), INVALID, "window"),
    (dict(c=cache(heads=3)), INVALID, "key heads"),
    (dict(q=operand(0, h=1000)), INVALID, "multiple of head_dim"),
    (dict(q=operand(0, h=1024, x=at(0) + 8)), INVALID, "16-byte"),
    (dict(q=operand(0, h=1024, ld_x=4100)), INVALID, "16-byte"),
    (dict(q=operand(0, h=1024, y=at(0))), INVALID, "overlaps"),
    (dict(q=operand(0, h=1024, y=at(30))), INVALID, "overlaps"),
    (dict(q=operand(0, h=1024, y=at(42))), INVALID, "overlaps"),
    (dict(b=batch(B=-1)), INVALID, "batch"),
    (dict(b=batch(max_q=0)), INVALID, "batch"),
    (dict(b=batch(max_len=0)), INVALID, "batch"),
    (dict(b=batch(ld_table=7)), INVALID, "batch"),
    (dict(b=batch(cu_q=None)), INVALID, "without cu_q"),
    (dict(b=batch(block_table=None)), INVALID, "block_table"),
    (dict(b=batch(seq_lens=at(41) + 2)), INVALID, "aligned"),
    (dict(b=batch(table_pages=1 << 30, ld_table=1 << 30)), UNSUPPORTED, "2^30"),
    (dict(b=batch(B=1 << 21)), UNSUPPORTED, "limits"),
    (dict(T=1 << 28), UNSUPPORTED, "too many"),
    (dict(T=1 << 20, b=batch(B=1 << 20, max_q=1 << 12)), UNSUPPORTED, "grid"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), ws=None), INVALID, "workspace"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), nb=64), INVALID, "workspace"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), ws=None, window=(1 << 63) - 1), INVALID, "workspace"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), ws=None, window=8191), INVALID, "workspace"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), ws=at(50) + 8), INVALID, "workspace"),
    (dict(b=batch(table_pages=512, ld_table=512, max_len=8192), ws=at(30)), INVALID, "overlaps"),
])
def test_attend_refusals(kw, code, text):
    assert call_attend(**kw) == code, message()
    assert text in message()


def test_calls_for_no_work():
    none = dict(x=None, y=None, gamma=None)
    assert call_rope(T=0, q=operand(0, **none), k=operand(5, **none), r=rope(cos_sin=None, positions=None)) == OK
    assert call_grad(T=0, ws=None, nb=0) == OK
    assert call_append(T=0, slots=None, c=cache(k=None, v=None, k_scales=None, v_scales=None)) == OK
    assert call_attend(T=0, b=batch(B=0), ws=None, nb=0) == OK
    assert call_attend(b=batch(B=0), ws=None, nb=0) == OK


def test_interleaved_caches_in_one_allocation_are_told_apart():
    """Pages that hold K, then V, in one allocation do not overlap; the same page does."""
    page = 4 * 16 * 64
    c = cache(k=at(30), v=at(30) + page, page_stride=2 * page)
    call_append(T=0, c=c)
    assert call_append(c=c, slots=None) == INVALID and "slots" in message()      # past the stride checks
    assert call_append(c=cache(k=at(30), v=at(30) + page - 16, page_stride=2 * page)) == INVALID
    assert "overlaps" in message()


def test_workspace_sizes():
    lib = qk.load_library()
    assert lib.qknorm_headwise_rope_backward_workspace(512, 512, 0, BF16, 128, 0) == 0
    assert lib.qknorm_headwise_rope_backward_workspace(500, 512, 10, BF16, 128, 0) == 0
    assert lib.qknorm_headwise_rope_backward_workspace(512, 512, 10, BF16, 128, 0) > 0
    assert lib.qknorm_paged_attend_workspace(1, 40, 8, 128, 1, 1, 64) == 0
    sizes = [lib.qknorm_paged_attend_workspace(1, 40, 8, 128, 1, 1, n) for n in range(64, 1 << 16, 777)]
    assert sizes == sorted(sizes) and sizes[-1] > 0     # never less for a longer cache
    assert lib.qknorm_paged_attend_workspace(1, 40, 7, 128, 1, 1, 4096) == 0
