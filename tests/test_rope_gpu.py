"""qknorm_headwise_rope and its backward pass on the GPU against the float64
oracle: row types, head widths that take each piece size, partial and
interleaved rotations, shared and per-head gamma, strides, in place, one
token to thousands, NaN and zero rows, positions outside the table."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


class Rows:
    """A case's rows inside wider buffers whose other columns hold canaries."""

    def __init__(self, seed, dtype, T, hq, hk, pad):
        r = C.rng(seed)
        self.dtype, self.hq, self.hk, self.pad = dtype, hq, hk, pad
        self.host = C.to_type(r.normal(size=(T, hq + pad + hk + pad)), dtype)
        self.t = C.dev(self.host)
        self.q, self.k = self.host[:, :hq], self.host[:, hq + pad:hq + pad + hk]
        self.qv, self.kv = self.views(self.t)

    def views(self, t):
        return t[:, :self.hq], t[:, self.hq + self.pad:self.hq + self.pad + self.hk]

    def rest_intact(self, t, before):
        keep = torch.ones(t.shape[1], dtype=torch.bool, device=t.device)
        keep[:self.hq] = False
        keep[self.hq + self.pad:self.hq + self.pad + self.hk] = False
        raw = t.view(torch.uint8).reshape(*t.shape, t.element_size())[:, keep]
        return torch.equal(raw, before.view(torch.uint8).reshape(*t.shape, t.element_size())[:, keep])


def _gammas(r, dtype, heads, d, stride):
    g = C.to_type(r.normal(1, 0.2, size=(heads - 1) * stride + d), "bf16" if dtype == "fp8" else dtype)
    return g, C.dev(g)


# dtype, T, heads_q, heads_k, head_dim, rot, interleaved, gamma stride (None: head_dim), row padding
CASES = [
    ("bf16", 1, 32, 32, 128, 128, False, 0, 0),
    ("bf16", 3, 5, 1, 128, 128, True, 0, 8),
    ("bf16", 257, 40, 8, 128, 128, False, 0, 128),
    ("bf16", 1500, 7, 3, 128, 64, False, None, 0),
    ("bf16", 700, 40, 8, 128, 32, True, 136, 16),
    ("bf16", 33, 6, 2, 64, 64, False, 0, 0),
    ("bf16", 65, 3, 3, 80, 80, False, 0, 0),       # 10 pieces of 16 bytes: 5 pairs on 8 lanes
    ("bf16", 65, 3, 3, 80, 40, False, 0, 0),       # 8-byte pieces
    ("bf16", 65, 3, 3, 80, 40, True, 84, 4),
    ("bf16", 50, 4, 2, 96, 96, False, 0, 1),       # odd strides: single elements
    ("bf16", 50, 4, 2, 256, 256, False, 0, 0),
    ("bf16", 9, 2, 1, 1024, 1024, False, 0, 0),
    ("bf16", 9, 2, 1, 1022, 510, True, 0, 0),      # 511 pairs on 64 lanes
    ("bf16", 21, 3, 2, 7, 4, False, 0, 0),         # odd head
    ("bf16", 21, 3, 2, 1, 0, False, 0, 0),
    ("bf16", 40, 4, 4, 128, 0, False, 0, 0),       # no rotation
    ("f32", 2047, 16, 4, 128, 64, True, None, 0),
    ("f32", 77, 3, 2, 128, 128, False, 0, 4),
    ("f32", 77, 3, 2, 100, 100, False, 0, 2),
    ("f32", 31, 3, 2, 33, 32, True, 0, 3),
    ("f32", 5, 2, 2, 1000, 998, False, 0, 0),
    ("fp8", 300, 10, 2, 128, 128, False, 0, 0),
    ("fp8", 300, 10, 2, 128, 64, True, 0, 16),
    ("fp8", 60, 3, 2, 80, 80, False, 0, 0),        # 8-byte pieces
    ("fp8", 60, 3, 2, 72, 36, False, 72, 5),
    ("fp8", 4500, 40, 8, 128, 128, False, 0, 0),
]


def _ids(c):
    return "-".join(str(x) for x in c)


def _setup(case, seed):
    dtype, T, nq, nk, d, rot, inter, stride, pad = case
    stride = d if stride is None else stride
    r = C.rng(seed)
    rows = Rows(seed + 1, dtype, T, nq * d, nk * d, pad)
    n_pos = 5000
    tab = C.table(n_pos, rot) if rot else None
    pos = r.integers(0, n_pos, T)
    if T > 2:
        pos[0], pos[-1] = 0, n_pos - 1
    cos, sin = O.angles(tab, pos, rot) if rot else (None, None)
    gq, gk = _gammas(r, dtype, nq, d, stride), _gammas(r, dtype, nk, d, stride)
    td = C.dev(tab) if rot else None
    pd = C.dev(pos) if rot else None
    return rows, stride, cos, sin, gq, gk, td, pd


@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_forward_against_the_oracle(case):
    dtype, T, nq, nk, d, rot, inter, _, pad = case
    print(f"[case] rope {case}", flush=True)
    rows, stride, cos, sin, gq, gk, td, pd = _setup(case, 11)
    out = C.dev(C.to_type(C.rng(5).normal(size=rows.host.shape), dtype))
    before = out.clone()
    oq, ok = rows.views(out)
    qk.qknorm_headwise_rope(rows.qv, rows.kv, gq[1], gk[1], EPS, d, td, pd, inter, stride, oq, ok)
    torch.cuda.synchronize()
    assert rows.rest_intact(out, before)
    assert C.same_bits(rows.t, C.dev(rows.host))
    for x, g, got in ((rows.q, gq[0], oq), (rows.k, gk[0], ok)):
        z = O.norm_rope(C.values(x), C.values(g), EPS, d, stride, None, None, False)
        want = z if cos is None else O.rotate(z, cos, sin, inter)
        if dtype == "fp8":
            want = np.clip(want, -448, 448)
        bound = C.rope_bound(z, cos, sin, inter, dtype)
        C.close(C.host_values(got).reshape(want.shape), want, bound, str(case))
    # in place gives the same bits
    qk.qknorm_headwise_rope(rows.qv, rows.kv, gq[1], gk[1], EPS, d, td, pd, inter, stride)
    torch.cuda.synchronize()
    assert C.same_bits(rows.qv, oq) and C.same_bits(rows.kv, ok)


@pytest.mark.parametrize("case", [c for c in CASES if c[0] != "fp8"], ids=_ids)
def test_backward_against_the_oracle(case):
    dtype, T, nq, nk, d, rot, inter, _, pad = case
    print(f"[case] rope backward {case}", flush=True)
    rows, stride, cos, sin, gq, gk, td, pd = _setup(case, 23)
    dy = Rows(77, dtype, T, nq * d, nk * d, pad)
    out = C.dev(C.to_type(C.rng(5).normal(size=rows.host.shape), dtype))
    before = out.clone()
    dxq, dxk = rows.views(out)
    got = qk.qknorm_headwise_rope_backward(dy.qv, dy.kv, rows.qv, rows.kv, gq[1], gk[1], EPS, d, td, pd, inter,
                                           stride, dx_q=dxq, dx_k=dxk)
    torch.cuda.synchronize()
    assert rows.rest_intact(out, before)
    assert C.same_bits(rows.t, C.dev(rows.host)) and C.same_bits(dy.t, C.dev(dy.host))
    for i, (x, g, w) in enumerate(((rows.q, dy.q, gq[0]), (rows.k, dy.k, gk[0]))):
        wx, wg, mx, mg = O.norm_rope_backward(C.values(x), C.values(g), C.values(w), EPS, d, stride, cos, sin, inter)
        # per term: the turned gradient within 3 u of its products' magnitudes, r within 32 u
        # (twice in the second term), the mean a chain of at most 32 products and 6 butterfly steps
        half = C.HALF[dtype] if dtype != "f32" else 0.0
        C.close(C.host_values(got[i]).reshape(wx.shape), wx, mx * 120 * C.U + np.abs(wx) * half + C.LOWEST[dtype],
                f"dx {i} {case}")
        # each term within 40 u; float32 sums over a wave's tokens, 8 waves and up to 64 lanes,
        # then float64 and one rounding
        C.close(got[2 + i].cpu().numpy().astype(np.float64), wg, mg * (40 + -(-T // 8) + 8 + 64 + 1) * C.U + 1e-30,
                f"dgamma {i} {case}")


def test_backward_repeats_bit_for_bit_and_in_place():
    case = ("bf16", 900, 10, 2, 128, 128, False, 0, 0)
    rows, stride, cos, sin, gq, gk, td, pd = _setup(case, 3)
    dy = Rows(78, "bf16", 900, 1280, 256, 0)
    args = (rows.qv, rows.kv, gq[1], gk[1], EPS, 128, td, pd)
    a = qk.qknorm_headwise_rope_backward(dy.qv, dy.kv, *args)
    b = qk.qknorm_headwise_rope_backward(dy.qv, dy.kv, *args)
    c = qk.qknorm_headwise_rope_backward(dy.qv, dy.kv, *args, dx_q=dy.qv, dx_k=dy.kv)
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert C.same_bits(x, y) and C.same_bits(x, z)
    dx = qk.qknorm_headwise_rope_backward(dy.qv, dy.kv, *args, need_dgamma=False)
    assert dx[2] is None and dx[3] is None


def test_gamma_gradient_leaves_gaps_between_heads_alone():
    d, stride, T = 64, 72, 40
    rows, _, cos, sin, gq, gk, td, pd = _setup(("f32", T, 4, 2, d, d, False, stride, 0), 9)
    dy = Rows(79, "f32", T, 4 * d, 2 * d, 0)
    dg = [torch.full_like(g[1], 7.5) for g in (gq, gk)]
    qk.qknorm_headwise_rope_backward(dy.qv, dy.kv, rows.qv, rows.kv, gq[1], gk[1], EPS, d, td, pd, False, stride,
                                     dgamma_q=dg[0], dgamma_k=dg[1])
    torch.cuda.synchronize()
    for t, heads in zip(dg, (4, 2)):
        for h in range(heads - 1):
            assert (t[h * stride + d:(h + 1) * stride] == 7.5).all()
            assert not (t[h * stride:h * stride + d] == 7.5).any()


def test_unusual_rows_and_positions():
    """A zero row gives zeros; NaN stays in its head; a position outside the table makes the
    rotated columns of its token NaN and nothing else."""
    T, d, rot = 6, 128, 64
    rows, stride, cos, sin, gq, gk, td, pd = _setup(("bf16", T, 4, 2, d, rot, False, 0, 0), 31)
    x = rows.t.clone()
    q, k = rows.views(x)
    q[1] = 0
    q[2, 5] = float("nan")
    q[3, d] = float("inf")
    pd = pd.clone()
    pd[4], pd[5] = -1, 5000
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    qk.qknorm_headwise_rope(q, k, gq[1], gk[1], EPS, d, td, pd, False, 0, oq, ok)
    torch.cuda.synchronize()
    o = oq.float().view(T, 4, d)
    assert (o[1] == 0).all()
    assert torch.isnan(o[2, 0]).all() and not torch.isnan(o[2, 1:]).any()
    assert not torch.isnan(o[3, 0]).any() and torch.isnan(o[3, 1]).any()
    for t in (4, 5):
        assert torch.isnan(o[t, :, :rot]).all() and not torch.isnan(o[t, :, rot:]).any()
        assert torch.isnan(ok.float().view(T, 2, d)[t, :, :rot]).all()


def test_without_rotation_is_the_headwise_call():
    case = ("bf16", 500, 8, 2, 128, 0, False, 0, 0)
    rows, _, _, _, gq, gk, _, _ = _setup(case, 8)
    a, b = torch.empty_like(rows.qv), torch.empty_like(rows.kv)
    c, d = torch.empty_like(rows.qv), torch.empty_like(rows.kv)
    qk.qknorm_headwise(rows.qv, rows.kv, gq[1], gk[1], EPS, 128, 0, a, b)
    qk.qknorm_headwise_rope(rows.qv, rows.kv, gq[1], gk[1], EPS, 128, None, None, out_q=c, out_k=d)
    torch.cuda.synchronize()
    # the sums run in another order: the roundings to bf16 may differ by one step at ties
    for x, y in ((a, c), (b, d)):
        assert (x.view(torch.int16).int() - y.view(torch.int16).int()).abs().max() <= 1


def test_rope_table_helper():
    t = qk.rope_table(70000, 64, base=1e6)
    want = C.table(70000, 64, base=1e6)
    # angles up to 7e4 formed in float64 on both sides: 7e4 * 2^-52 apart at most, then one rounding
    assert np.abs(t.cpu().numpy().astype(np.float64) - want).max() <= 2.0 ** -23
    f = torch.rand(8, dtype=torch.float64)
    t = qk.rope_table(10, 16, inv_freq=f).cpu()
    assert torch.allclose(t[3, :8].double(), torch.cos(3 * f), atol=1e-7)


def test_marshalling_refusals():
    rows, _, _, _, gq, gk, td, pd = _setup(("bf16", 8, 4, 2, 128, 128, False, 0, 0), 8)
    ok = (rows.qv, rows.kv, gq[1], gk[1], EPS, 128, td, pd)

    def refused(i, value, error):
        a = list(ok)
        a[i] = value
        with pytest.raises(error):
            qk.qknorm_headwise_rope(*a)

    refused(0, rows.qv[:4], ValueError)
    refused(2, gq[1][:100], ValueError)
    refused(2, gq[1].float(), ValueError)
    refused(2, None, ValueError)
    refused(6, td.double(), ValueError)
    refused(6, td.cpu(), ValueError)
    refused(7, pd[:4], ValueError)
    refused(7, pd.int(), ValueError)
    refused(7, pd.cpu(), ValueError)
    refused(5, 96, qk.QKNormError)
    with pytest.raises(ValueError):
        qk.qknorm_headwise_rope(*ok, out_q=torch.empty_like(rows.qv, dtype=torch.float32))
