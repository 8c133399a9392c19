"""Quantised appends of normalised keys that hold infinities and NaN, against the float64 oracle:
a head with an infinity has the factor 0, so the infinity (and its partner in the rotation) is NaN
and everything else of the head 0; blocks that hold neither keep finite codes."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O
from test_paged_append_gpu import EPS, Case, _at

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


CASES = [     # one chunk of a head a lane, from one to four slots a wave; the last three: the layout of pairs
    dict(dtype="bf16", T=40, nq=4, nk=2, d=128, rot=128, inter=False),
    dict(dtype="bf16", T=40, nq=4, nk=2, d=128, rot=64, inter=True),
    dict(dtype="bf16", T=40, nq=4, nk=2, d=128, rot=0, inter=False),
    dict(dtype="bf16", T=1000, nq=12, nk=12, d=128, rot=128, inter=False),
    dict(dtype="f32", T=40, nq=2, nk=3, d=64, rot=32, inter=False),
    dict(dtype="f32", T=40, nq=2, nk=1, d=256, rot=256, inter=True, stride=256),
    dict(dtype="bf16", T=40, nq=4, nk=2, d=96, rot=96, inter=False),
    dict(dtype="f32", T=40, nq=4, nk=2, d=96, rot=64, inter=True),
    dict(dtype="bf16", T=1400, nq=12, nk=6, d=96, rot=96, inter=False),
]


def _name(k):
    return "-".join(str(v) for v in k.values())


def _special(c):
    """Puts infinities and NaN into some heads of Q and K: one element, two of both signs, the
    first and the last column, a whole head."""
    x = C.values(c.host).copy()
    d = c.d
    for side, heads in ((0, c.nq), (1, c.nk)):
        at = c.cut[side] + (heads - 1) * d            # the side's last head
        for t, cols, value in ((5, [d // 2 + 3], np.inf), (6, [1], -np.inf), (7, [d - 1], np.inf), (8, [0], np.nan),
                               (9, range(d), np.inf), (10, [40], 3.0e38)):
            x[t, [at + i for i in cols]] = value
        x[11, at + 2], x[11, at + d - 2] = np.inf, -np.inf
        x[12, at + 2], x[12, at + d - 2] = np.inf, np.nan
    if c.dtype == "f32":
        c.host = x.astype(np.float32)
    else:
        keep = np.isfinite(x)
        bits = C.to_type(np.where(keep, x, 0.0), "bf16")
        c.host = np.where(keep, bits, np.where(np.isnan(x), 0x7FC0, np.where(x > 0, 0x7F80, 0xFF80))).astype(np.uint16)
    c.t = C.dev(c.host)
    c.q, c.k, c.v = (c.t[:, a:b] for a, b in zip(c.cut, c.cut[1:]))
    c.hq, c.hk, c.hv = (C.values(c.host[:, a:b]) for a, b in zip(c.cut, c.cut[1:]))
    assert np.isinf(c.hk).any() and np.isnan(c.hk).any()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("kw,several_axes", [(k, a) for k in CASES for a in (False, True) if k["rot"] or not a],
                         ids=lambda v: _name(v) if isinstance(v, dict) else "axes" if v else "one axis")
def test_normalised_keys(fmt, kw, several_axes):
    print(f"[case] infinite keys {fmt} {kw} axes={several_axes}", flush=True)
    c = Case(61, **kw)
    _special(c)
    last = c.d if fmt == "mxfp8" else c.d // 2
    kc, vc = (torch.zeros((c.pages, c.nk, c.ps, last), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((c.pages, c.nk, c.ps, c.d // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    dt = C.TORCH[c.dtype]
    out_q = torch.full((c.T, c.nq * c.d), 3.0, dtype=dt, device="cuda")
    out_k = torch.full((c.T, c.nk * c.d), 5.0, dtype=dt, device="cuda")
    slots = C.dev(c.slots)
    args = (c.q, c.k, c.v, *c.gt, EPS, c.d, c.table)
    more = dict(k_scales=ks, v_scales=vs, interleaved=c.inter, gamma_head_stride=c.stride, out_q=out_q, out_k=out_k)
    if several_axes:
        axes = qk.rope_axes((kw["rot"] // 4, kw["rot"] // 2 - kw["rot"] // 4))
        pos = C.rng(3).integers(0, 4000, (2, c.T))
        c.cos, c.sin = O.axis_angles(c.table.cpu().numpy(), pos, axes, kw["rot"])
        qk.qknorm_paged_append_axes(*args, C.dev(pos), axes, kc, vc, slots, **more)
    else:
        qk.qknorm_paged_append(*args, c.pos, kc, vc, slots, **more)
    back = qk.qknorm_paged_gather(kc, vc, slots, c.d, ks, vs, dtype=dt)[0]
    torch.cuda.synchronize()
    s = c.slots[c.keep]
    with np.errstate(invalid="ignore"):
        keys, (_, queries) = c.keys()[c.keep], c.queries()
    codes, scales, values = (O.mxfp8_quantize if fmt == "mxfp8" else O.mxfp4_quantize)(keys)
    got = _at(ks.cpu().numpy(), s, c.ps)
    assert np.array_equal(got, scales), f"{int((got != scales).sum())} scales of {scales.size}"
    held = _at(kc.cpu().numpy(), s, c.ps)
    if fmt == "mxfp8":        # only the sign of a zero may differ
        assert ((held == codes) | ((held & 127) + (codes & 127) == 0)).all()
    else:
        for a, b in ((held & 15, codes & 15), (held >> 4, codes >> 4)):
            assert ((a == b) | ((a & 7) + (b & 7) == 0)).all()
    for rows in (out_k, back):
        assert np.array_equal(C.host_values(rows).reshape(c.T, c.nk, c.d)[c.keep], values, equal_nan=True)
    # The call's queries follow the same formula, in float32: where the squares of finite elements
    # pass its range (token 10: 9e76) the factor is 0, and 3e38 gamma may be infinite.
    got, rows = C.host_values(out_q).reshape(c.T, c.nq, c.d), c.keep & (np.arange(c.T) != 10)
    assert np.array_equal(np.isnan(got[rows]), np.isnan(queries[rows]))
