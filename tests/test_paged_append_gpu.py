"""qknorm_paged_append on the GPU against the float64 oracle: row-type and
MXFP4 caches, layouts, padded rows, and that nothing else is written."""

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


class Case:
    def __init__(self, seed, dtype, T, nq, nk, d, rot, inter, norm=True, stride=0, pad=0, pages=None, ps=16,
                 n_pos=4000, spread=False):
        r = C.rng(seed)
        self.T, self.nq, self.nk, self.d, self.inter, self.stride, self.dtype = T, nq, nk, d, inter, stride, dtype
        x = r.normal(size=(T, (nq + 2 * nk) * d + pad))
        if spread:      # magnitudes over many binades
            x *= np.exp(r.normal(size=(T, 1)) * 6)
        self.host = C.to_type(x, dtype)
        self.t = C.dev(self.host)
        self.cut = (0, nq * d, (nq + nk) * d, (nq + 2 * nk) * d)
        self.q, self.k, self.v = (self.t[:, a:b] for a, b in zip(self.cut, self.cut[1:]))
        self.hq, self.hk, self.hv = (C.values(self.host[:, a:b]) for a, b in zip(self.cut, self.cut[1:]))
        tab = C.table(n_pos, rot) if rot else None
        pos = r.integers(0, n_pos, T)
        self.cos, self.sin = O.angles(tab, pos, rot) if rot else (None, None)
        self.table, self.pos = (C.dev(tab), C.dev(pos)) if rot else (None, None)
        g = [C.to_type(r.normal(1, 0.2, size=(n - 1) * stride + d), dtype) for n in (nq, nk)]
        self.g = [C.values(x) if norm else None for x in g]
        self.gt = [C.dev(x) if norm else None for x in g]
        self.ps, self.pages = ps, pages or (T // ps + 3)
        self.slots = r.permutation(self.pages * ps)[:T].astype(np.int64)
        if T > 4:
            self.slots[[1, T - 1]] = -1
            self.slots[2] = self.pages * ps + 5     # past the last page: passed over as well
        self.keep = (self.slots >= 0) & (self.slots < self.pages * ps)

    def keys(self):
        return O.norm_rope(self.hk, self.g[1], EPS, self.d, self.stride, self.cos, self.sin, self.inter)

    def queries(self):
        z = O.norm_rope(self.hq, self.g[0], EPS, self.d, self.stride, None, None, self.inter)
        return z, z if self.cos is None else O.rotate(z, self.cos, self.sin, self.inter)

    def check_q(self, out, before):
        z, want = self.queries()
        got = C.host_values(out).reshape(want.shape)
        bound = C.rope_bound(z, self.cos, self.sin, self.inter, self.dtype)
        C.close(got[self.keep], want[self.keep], bound[self.keep], "q")
        assert C.same_bits(out[torch.from_numpy(~self.keep).cuda()], before[torch.from_numpy(~self.keep).cuda()])


def _at(cache, slots, ps):
    """The entries of [pages, heads, ps, n] at slots: [T, heads, n]."""
    return cache[slots // ps, :, slots % ps]


MX = [
    dict(dtype="bf16", T=1, nq=40, nk=8, d=128, rot=128, inter=False),
    dict(dtype="bf16", T=64, nq=40, nk=8, d=128, rot=128, inter=False),
    dict(dtype="bf16", T=1000, nq=10, nk=2, d=128, rot=128, inter=True, ps=64),
    dict(dtype="bf16", T=300, nq=7, nk=7, d=128, rot=64, inter=False, norm=False, ps=128),
    dict(dtype="bf16", T=129, nq=8, nk=4, d=64, rot=32, inter=False, pad=8),
    dict(dtype="bf16", T=90, nq=4, nk=2, d=96, rot=96, inter=False),
    dict(dtype="bf16", T=90, nq=4, nk=2, d=32, rot=16, inter=True),
    dict(dtype="bf16", T=50, nq=4, nk=2, d=256, rot=256, inter=False, stride=256),
    dict(dtype="bf16", T=50, nq=4, nk=2, d=1024, rot=512, inter=False),
    dict(dtype="bf16", T=50, nq=4, nk=2, d=160, rot=100, inter=False, pad=3),   # single elements
    dict(dtype="bf16", T=40, nq=2, nk=2, d=992, rot=990, inter=False, pad=1),
    dict(dtype="f32", T=77, nq=6, nk=3, d=128, rot=128, inter=False),
    dict(dtype="f32", T=77, nq=6, nk=3, d=64, rot=64, inter=True, norm=False, pad=2),
    dict(dtype="bf16", T=200, nq=4, nk=4, d=128, rot=0, inter=False, norm=False, spread=True),
    dict(dtype="bf16", T=4500, nq=40, nk=8, d=128, rot=128, inter=False, ps=32),
]


@pytest.mark.parametrize("kw", MX, ids=lambda k: "-".join(str(v) for v in k.values()))
@pytest.mark.parametrize("rows_out", [True, False])
def test_mxfp4(kw, rows_out):
    print(f"[case] append mxfp4 {kw}", flush=True)
    c = Case(17, **kw)
    dt = C.TORCH[c.dtype]
    r = np.random.default_rng(1)
    shape = (c.pages, c.nk, c.ps)
    fill = [r.integers(0, 256, shape + (n,), dtype=np.uint8) for n in (c.d // 2, c.d // 2, c.d // 32, c.d // 32)]
    kc, vc, ks, vs = (torch.from_numpy(f.copy()).cuda() for f in fill)
    out_q = torch.full((c.T, c.nq * c.d), 3.0, dtype=dt, device="cuda")
    rows = [torch.full((c.T, c.nk * c.d), 5.0, dtype=dt, device="cuda") if rows_out else None for _ in range(2)]
    before_q = out_q.clone()
    qk.qknorm_paged_append(c.q, c.k, c.v, *c.gt, EPS, c.d, c.table, c.pos, kc, vc, C.dev(c.slots), ks, vs, c.inter,
                           c.stride, out_q=out_q, out_k=rows[0], out_v=rows[1])
    torch.cuda.synchronize()
    assert C.same_bits(c.t, C.dev(c.host))
    c.check_q(out_q, before_q)
    s = c.slots[c.keep]
    for codes, scales, f_codes, f_scales, want, out in ((kc, ks, fill[0], fill[2], c.keys(), rows[0]),
                                                        (vc, vs, fill[1], fill[3],
                                                         c.hv.reshape(c.T, c.nk, c.d), rows[1])):
        w_codes, w_scales, w_values = O.mxfp4_quantize(want[c.keep])
        f_codes, f_scales = f_codes.copy(), f_scales.copy()
        f_codes[s // c.ps, :, s % c.ps] = w_codes
        f_scales[s // c.ps, :, s % c.ps] = w_scales
        got_codes, got_scales = codes.cpu().numpy(), scales.cpu().numpy()
        assert np.array_equal(got_scales, f_scales)          # every scale, and no other place written
        # codes too; only the sign of a zero may differ, where a key's rotation cancels to zero
        for got, want in ((got_codes & 15, f_codes & 15), (got_codes >> 4, f_codes >> 4)):
            assert ((got == want) | ((got & 7) + (want & 7) == 0)).all()
        if out is not None:
            got = C.host_values(out).reshape(c.T, c.nk, c.d)
            assert np.array_equal(got[c.keep], w_values)
            assert (got[~c.keep] == 5.0).all()


ROWS = [
    dict(dtype="bf16", T=64, nq=32, nk=32, d=128, rot=128, inter=False, norm=False),
    dict(dtype="bf16", T=999, nq=10, nk=2, d=128, rot=64, inter=True, ps=1),
    dict(dtype="bf16", T=50, nq=4, nk=2, d=80, rot=80, inter=False, ps=8),
    dict(dtype="bf16", T=50, nq=4, nk=2, d=33, rot=32, inter=False, pad=1),
    dict(dtype="f32", T=77, nq=6, nk=3, d=128, rot=128, inter=False, stride=128),
]


@pytest.mark.parametrize("kw", ROWS, ids=lambda k: "-".join(str(v) for v in k.values()))
@pytest.mark.parametrize("layout", ["heads first", "tokens first", "one allocation"])
def test_row_type(kw, layout):
    print(f"[case] append rows {kw} {layout}", flush=True)
    c = Case(19, **kw)
    dt = C.TORCH[c.dtype]
    if layout == "heads first":
        kc, vc = (torch.full((c.pages, c.nk, c.ps, c.d), 9.0, dtype=dt, device="cuda") for _ in range(2))
    elif layout == "tokens first":
        kc, vc = (torch.full((c.pages, c.ps, c.nk, c.d), 9.0, dtype=dt, device="cuda").transpose(1, 2)
                  for _ in range(2))
    else:
        both = torch.full((c.pages, 2, c.nk, c.ps, c.d), 9.0, dtype=dt, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    out_k = torch.full((c.T, c.nk * c.d), 5.0, dtype=dt, device="cuda")
    qk.qknorm_paged_append(c.q, c.k, c.v, *c.gt, EPS, c.d, c.table, c.pos, kc, vc, C.dev(c.slots),
                           interleaved=c.inter, gamma_head_stride=c.stride, out_k=out_k)       # q in place
    torch.cuda.synchronize()
    c.check_q(c.q, C.dev(c.host)[:, :c.nq * c.d])
    s = c.slots[c.keep]
    z = O.norm_rope(c.hk, c.g[1], EPS, c.d, c.stride, None, None, c.inter)
    bound = C.rope_bound(z, c.cos, c.sin, c.inter, c.dtype)
    kh, vh = C.host_values(kc), C.host_values(vc)
    C.close(_at(kh, s, c.ps), c.keys()[c.keep], bound[c.keep], "k")
    assert np.array_equal(_at(vh, s, c.ps), c.hv.reshape(c.T, c.nk, c.d)[c.keep])
    got = C.host_values(out_k).reshape(c.T, c.nk, c.d)
    assert np.array_equal(got[c.keep], _at(kh, s, c.ps)) and (got[~c.keep] == 5.0).all()
    free = np.ones(c.pages * c.ps, bool)
    free[s] = False
    f = np.nonzero(free)[0]
    assert (_at(kh, f, c.ps) == 9.0).all() and (_at(vh, f, c.ps) == 9.0).all()


def test_values_that_are_not_finite_mark_their_blocks():
    c = Case(23, "bf16", 20, 2, 2, 128, 128, False, norm=False)
    c.slots = np.arange(20)
    v = c.v.clone()
    v[3, 5] = float("inf")
    v[4, 128 + 40] = float("nan")
    v[5, :] = 0
    v[6, 0:32] = -0.0
    kc = torch.zeros((2, 2, 16, 64), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((2, 2, 16, 4), dtype=torch.uint8, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    out_v = torch.empty_like(v)
    qk.qknorm_paged_append(None, c.k, v, None, None, EPS, 128, c.table, c.pos, kc, vc, C.dev(c.slots), ks, vs,
                           out_v=out_v)
    torch.cuda.synchronize()
    sc = _at(vs.cpu().numpy(), c.slots, 16)
    bad = np.zeros_like(sc, bool)
    bad[3, 0, 0] = bad[4, 1, 1] = True
    assert np.array_equal(sc == 255, bad)
    assert (sc[5] == 27).all() and sc[6, 0, 0] == 27
    o = out_v.float().cpu().numpy().reshape(20, 2, 4, 32)
    assert np.isnan(o[bad]).all() and not np.isnan(o[~bad]).any() and (o[5] == 0).all()


def test_appending_keys_and_values_alone_leaves_queries_out():
    c = Case(29, "bf16", 70, 8, 2, 128, 128, False)
    a = [torch.zeros((c.pages, 2, 16, 64), dtype=torch.uint8, device="cuda") for _ in range(4)]
    s = [torch.zeros((c.pages, 2, 16, 4), dtype=torch.uint8, device="cuda") for _ in range(4)]
    slots = C.dev(c.slots)
    assert qk.qknorm_paged_append(None, c.k, c.v, None, c.gt[1], EPS, 128, c.table, c.pos, a[0], a[1], slots, s[0],
                                  s[1]) is None
    qk.qknorm_paged_append(c.q, c.k, c.v, *c.gt, EPS, 128, c.table, c.pos, a[2], a[3], slots, s[2], s[3],
                           out_q=torch.empty_like(c.q))
    torch.cuda.synchronize()
    for x, y in ((a[0], a[2]), (a[1], a[3]), (s[0], s[2]), (s[1], s[3])):
        assert torch.equal(x, y)


def test_marshalling_refusals():
    c = Case(31, "bf16", 8, 4, 2, 128, 128, False)
    kc = torch.zeros((3, 2, 16, 64), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((3, 2, 16, 4), dtype=torch.uint8, device="cuda")
    kw = dict(k_cache=kc, v_cache=kc.clone(), slots=C.dev(c.slots), k_scales=ks, v_scales=ks.clone())

    def call(**over):
        a = {**kw, **over}
        qk.qknorm_paged_append(c.q, c.k, c.v, *c.gt, EPS, 128, c.table, c.pos, **a)

    for over in (dict(k_scales=None), dict(k_cache=kc[:2]), dict(k_cache=kc.bfloat16()), dict(slots=kw["slots"].int()),
                 dict(slots=kw["slots"][:3]), dict(k_scales=ks[..., :2]), dict(v_scales=ks.cpu()),
                 dict(k_cache=kc[..., :32])):
        with pytest.raises(ValueError):
            call(**over)
    with pytest.raises(qk.QKNormError):
        call(v_cache=kc)        # k and v in one place
