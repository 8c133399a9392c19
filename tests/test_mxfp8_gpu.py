"""MXFP8 caches on the GPU against the float64 oracle: the append that writes them (codes and
scales are those of exact arithmetic, nothing else is written), with one and several axes, and
qknorm_paged_gather, which reads caches of every format back."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O
from test_paged_append_gpu import EPS, MX, ROWS, Case, _at

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


def _name(k):
    return "-".join(str(v) for v in k.values()) if isinstance(k, dict) else str(k)


MORE = [     # three and four slots to a wave, partners 32 lanes apart, the layout of pairs with three slots
    dict(dtype="bf16", T=1000, nq=12, nk=12, d=128, rot=128, inter=False),
    dict(dtype="bf16", T=700, nq=16, nk=16, d=128, rot=128, inter=True, ps=64),
    dict(dtype="f32", T=700, nq=8, nk=8, d=128, rot=128, inter=False, stride=128),
    dict(dtype="bf16", T=1400, nq=12, nk=6, d=96, rot=96, inter=False),
    dict(dtype="f32", T=1400, nq=8, nk=4, d=96, rot=96, inter=True),
    dict(dtype="f32", T=50, nq=3, nk=2, d=256, rot=256, inter=False),
]


def _same_codes(got, want):
    """Only the sign of a zero may differ, where a key's rotation cancels to zero."""
    return ((got == want) | ((got & 127) + (want & 127) == 0)).all()


@pytest.mark.parametrize("kw", MX + MORE, ids=_name)
@pytest.mark.parametrize("rows_out,layout", [(True, "heads first"), (False, "tokens first")])
def test_append(kw, rows_out, layout):
    print(f"[case] append mxfp8 {kw} {layout}", flush=True)
    c = Case(17, **kw)
    dt = C.TORCH[c.dtype]
    r = np.random.default_rng(1)
    fill = [r.integers(0, 256, (c.pages, c.nk, c.ps, n), dtype=np.uint8) for n in (c.d, c.d, c.d // 32, c.d // 32)]
    kc, vc, ks, vs = (torch.from_numpy(f.copy()).cuda() for f in fill)
    if layout == "tokens first":
        kc, vc = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kc, vc))
    out_q = torch.full((c.T, c.nq * c.d), 3.0, dtype=dt, device="cuda")
    rows = [torch.full((c.T, c.nk * c.d), 5.0, dtype=dt, device="cuda") if rows_out else None for _ in range(2)]
    before_q = out_q.clone()
    slots = C.dev(c.slots)
    qk.qknorm_paged_append(c.q, c.k, c.v, *c.gt, EPS, c.d, c.table, c.pos, kc, vc, slots, ks, vs, c.inter, c.stride,
                           out_q=out_q, out_k=rows[0], out_v=rows[1])
    back = qk.qknorm_paged_gather(kc, vc, slots, c.d, ks, vs, dtype=torch.float32)
    torch.cuda.synchronize()
    assert C.same_bits(c.t, C.dev(c.host))
    c.check_q(out_q, before_q)
    s = c.slots[c.keep]
    for codes, scales, f_codes, f_scales, want, out, got_rows in (
            (kc, ks, fill[0], fill[2], c.keys(), rows[0], back[0]),
            (vc, vs, fill[1], fill[3], c.hv.reshape(c.T, c.nk, c.d), rows[1], back[1])):
        w_codes, w_scales, w_values = O.mxfp8_quantize(want[c.keep])
        f_codes, f_scales = f_codes.copy(), f_scales.copy()
        f_codes[s // c.ps, :, s % c.ps] = w_codes
        f_scales[s // c.ps, :, s % c.ps] = w_scales
        assert np.array_equal(scales.cpu().numpy(), f_scales)          # every scale, and no other place written
        assert _same_codes(codes.cpu().numpy(), f_codes)
        if out is not None:
            got = C.host_values(out).reshape(c.T, c.nk, c.d)
            assert np.array_equal(got[c.keep], w_values)
            assert (got[~c.keep] == 5.0).all()
        got = got_rows.double().cpu().numpy().reshape(c.T, c.nk, c.d)
        assert np.array_equal(got[c.keep], w_values) and not got[~c.keep].any()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "rows"])
@pytest.mark.parametrize("kw", [
    dict(dtype="bf16", T=600, nq=10, nk=2, d=128, rot=128, inter=False),
    dict(dtype="bf16", T=33, nq=3, nk=2, d=128, rot=64, inter=True, norm=False),
    dict(dtype="f32", T=200, nq=4, nk=4, d=64, rot=64, inter=False),
    dict(dtype="bf16", T=1200, nq=12, nk=6, d=96, rot=96, inter=False),
], ids=_name)
@pytest.mark.parametrize("spread", [False, True])
def test_append_with_several_axes(fmt, kw, spread):
    print(f"[case] append axes {fmt} {kw} {spread}", flush=True)
    c = Case(37, **kw)
    n = kw["rot"] // 2
    axes = qk.rope_axes((n // 4, (n - n // 4 + 1) // 2, (n - n // 4) // 2), spread)
    pos = C.rng(3).integers(0, 4000, (3, c.T))
    c.cos, c.sin = O.axis_angles(c.table.cpu().numpy(), pos, axes, kw["rot"])
    dt = C.TORCH[c.dtype]
    last = {"mxfp8": c.d, "mxfp4": c.d // 2, "rows": c.d}[fmt]
    kc, vc = (torch.zeros((c.pages, c.nk, c.ps, last), dtype=dt if fmt == "rows" else torch.uint8, device="cuda")
              for _ in range(2))
    ks, vs = (None if fmt == "rows" else torch.zeros((c.pages, c.nk, c.ps, c.d // 32), dtype=torch.uint8, device="cuda")
              for _ in range(2))
    out_q = torch.full((c.T, c.nq * c.d), 3.0, dtype=dt, device="cuda")
    before_q = out_q.clone()
    qk.qknorm_paged_append_axes(c.q, c.k, c.v, *c.gt, EPS, c.d, c.table, C.dev(pos), axes, kc, vc, C.dev(c.slots), ks,
                                vs, c.inter, c.stride, out_q=out_q)
    torch.cuda.synchronize()
    c.check_q(out_q, before_q)
    s, want = c.slots[c.keep], c.keys()[c.keep]
    if fmt == "rows":
        z = O.norm_rope(c.hk, c.g[1], EPS, c.d, c.stride, None, None, c.inter)
        C.close(_at(C.host_values(kc), s, c.ps), want, C.rope_bound(z, c.cos, c.sin, c.inter, c.dtype)[c.keep], "k")
        return
    codes, scales, _ = (O.mxfp8_quantize if fmt == "mxfp8" else O.mxfp4_quantize)(want)
    assert np.array_equal(_at(ks.cpu().numpy(), s, c.ps), scales)
    got = _at(kc.cpu().numpy(), s, c.ps)
    if fmt == "mxfp8":
        assert _same_codes(got, codes)
    else:
        for a, b in ((got & 15, codes & 15), (got >> 4, codes >> 4)):
            assert ((a == b) | ((a & 7) + (b & 7) == 0)).all()


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("gammas", ["ordinary", "far", "none"])
@pytest.mark.parametrize("dtype,d,rot,inter", [("bf16", 128, 128, False), ("bf16", 128, 64, True), ("f32", 128, 128, False),
                                               ("f32", 256, 256, False), ("bf16", 96, 96, False)])
def test_keys_far_from_one(dtype, d, rot, inter, gammas, eps):
    """Sums, factors or products beyond float32's normal range: codes and scales are still those
    of exact arithmetic."""
    print(f"[case] key codes {dtype} {d} {gammas} {eps}", flush=True)
    r = C.rng(d + rot)
    T, heads, ps = 256, 2, 16
    scale = 2.0 ** np.linspace(-132, 123, T)[r.permutation(T)][:, None]
    host = C.to_type(np.clip(r.normal(size=(T, heads * d)) * scale, -3e38, 3e38), dtype)
    v = C.to_type(np.clip(r.normal(size=(T, heads * d)) * scale, -3e38, 3e38), dtype)
    g = r.normal(1, 0.2, size=d)
    if gammas == "far":
        g = g * 2.0 ** r.integers(-90, 90, d)
    g = None if gammas == "none" else C.to_type(g, dtype)
    tab, pos = C.table(300, rot), r.integers(0, 300, T)
    pages = -(-T // ps)
    kc, vc = (torch.zeros((pages, heads, ps, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, heads, ps, d // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = np.arange(T, dtype=np.int64)
    qk.qknorm_paged_append(None, C.dev(host), C.dev(v), None, None if g is None else C.dev(g), eps, d, C.dev(tab),
                           C.dev(pos), kc, vc, C.dev(slots), ks, vs, inter)
    torch.cuda.synchronize()
    cos, sin = O.angles(tab, pos, rot)
    with np.errstate(all="ignore"):
        keys = O.norm_rope(C.values(host), None if g is None else C.values(g), eps, d, 0, cos, sin, inter)
    for what, want, c, s in (("k", keys, kc, ks), ("v", C.values(v).reshape(T, heads, d), vc, vs)):
        codes, scales, _ = O.mxfp8_quantize(want)
        got = _at(s.cpu().numpy(), slots, ps)
        assert np.array_equal(got, scales), f"{what}: {int((got != scales).sum())} scales of {scales.size}"
        assert _same_codes(_at(c.cpu().numpy(), slots, ps), codes), what


def test_values_that_are_not_finite_mark_their_blocks():
    c = Case(23, "bf16", 20, 2, 2, 128, 128, False, norm=False)
    c.slots = np.arange(20)
    v = c.v.clone()
    v[3, 5] = float("inf")
    v[4, 128 + 40] = float("nan")
    v[5, :] = 0
    v[6, 0:32] = -0.0
    v[7, 0:32] = torch.finfo(torch.bfloat16).max
    kc = torch.zeros((2, 2, 16, 128), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((2, 2, 16, 4), dtype=torch.uint8, device="cuda")
    vc, vs = kc.clone(), ks.clone()
    out_v = torch.empty_like(v)
    qk.qknorm_paged_append(None, c.k, v, None, None, EPS, 128, c.table, c.pos, kc, vc, C.dev(c.slots), ks, vs,
                           out_v=out_v)
    back = qk.qknorm_paged_gather(kc, vc, C.dev(c.slots), 128, ks, vs)
    torch.cuda.synchronize()
    sc = _at(vs.cpu().numpy(), c.slots, 16)
    bad = np.zeros_like(sc, bool)
    bad[3, 0, 0] = bad[4, 1, 1] = True
    assert np.array_equal(sc == 255, bad)
    assert (sc[5] == 27).all() and sc[6, 0, 0] == 27 and sc[7, 0, 0] == 246
    assert back[1].dtype == torch.bfloat16
    for rows in (out_v, back[1]):
        o = rows.float().cpu().numpy().reshape(20, 2, 4, 32)
        assert np.isnan(o[bad]).all() and not np.isnan(o[~bad]).any() and (o[5] == 0).all()
        assert (o[7, 0, 0] == 448 * 2.0 ** 119).all()


# ------------------------------------------------------------------ reading back
def _codes_cache(r, fmt, pages, heads, ps, d):
    codes = [r.integers(0, 256, (pages, heads, ps, d // 2 if fmt == "mxfp4" else d), dtype=np.uint8) for _ in range(2)]
    scales = [r.integers(20, 256, (pages, heads, ps, d // 32), dtype=np.uint8) for _ in range(2)]
    return codes, scales


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,heads,d,ps,pad", [(1, 1, 32, 16, 0), (700, 8, 128, 16, 0), (333, 3, 96, 64, 8),
                                              (50, 2, 1024, 32, 0), (257, 5, 64, 16, 3)])
def test_gather_codes(fmt, dtype, T, heads, d, ps, pad):
    """Every byte of codes and scales, the NaN ones among them; slots twice, negative and past the end."""
    print(f"[case] gather {fmt} {dtype} {T} {heads} {d}", flush=True)
    r = C.rng(T + d)
    pages = T // ps + 2
    codes, scales = _codes_cache(r, fmt, pages, heads, ps, d)
    slots = r.integers(0, pages * ps, T).astype(np.int64)
    if T > 4:
        slots[[1, T - 1]] = -1
        slots[2] = pages * ps
        slots[3] = slots[4]
    keep = (slots >= 0) & (slots < pages * ps)
    dt = C.TORCH[dtype]
    out = [torch.full((T, heads * d + pad), 3.0, dtype=dt, device="cuda") for _ in range(2)]
    views = [o[:, :heads * d] for o in out]
    dev = [torch.from_numpy(x).cuda() for x in codes + scales]
    qk.qknorm_paged_gather(dev[0], dev[1], C.dev(slots), d, dev[2], dev[3], *views)
    only_v = torch.full_like(views[1], 3.0)
    assert qk.qknorm_paged_gather(dev[0], dev[1], C.dev(slots), d, dev[2], dev[3], out_v=only_v)[0] is None
    torch.cuda.synchronize()
    assert C.same_bits(only_v, views[1].contiguous())
    value = O.mxfp4_values if fmt == "mxfp4" else O.mxfp8_values
    for i in range(2):
        want = value(_at(codes[i], slots[keep], ps), _at(scales[i], slots[keep], ps))
        got = C.host_values(views[i]).reshape(T, heads, d)
        # exact: scale bytes from 20 on, so the least value is 2^-9 2^-107
        assert np.array_equal(got[keep], want, equal_nan=True)
        assert (got[~keep] == 3.0).all() and (out[i][:, heads * d:] == 3.0).all()


@pytest.mark.parametrize("kw", ROWS, ids=_name)
@pytest.mark.parametrize("layout", ["heads first", "tokens first", "one allocation"])
def test_gather_rows_is_the_inverse_of_the_append(kw, layout):
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
    ok, ov = (torch.zeros((c.T, c.nk * c.d), dtype=dt, device="cuda") for _ in range(2))
    slots = C.dev(c.slots)
    qk.qknorm_paged_append(c.q, c.k, c.v, *c.gt, EPS, c.d, c.table, c.pos, kc, vc, slots, interleaved=c.inter,
                           gamma_head_stride=c.stride, out_k=ok, out_v=ov)
    k, v = qk.qknorm_paged_gather(kc, vc, slots, c.d)
    torch.cuda.synchronize()
    assert k.dtype == dt and C.same_bits(k, ok) and C.same_bits(v, ov)


def test_gather_of_nothing_and_marshalling_refusals():
    kc = torch.zeros((3, 2, 16, 128), dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks = torch.zeros((3, 2, 16, 4), dtype=torch.uint8, device="cuda")
    vs = ks.clone()
    slots = torch.arange(5, device="cuda")
    k, v = qk.qknorm_paged_gather(kc, vc, slots[:0], 128, ks, vs)
    assert k.shape == (0, 256) and v.shape == (0, 256)
    out = torch.zeros((5, 256), dtype=torch.bfloat16, device="cuda")
    for a, kw in (((kc, vc, slots.int(), 128, ks, vs), {}), ((kc, vc, slots.cpu(), 128, ks, vs), {}),
                  ((kc, vc, slots, 128, ks, None), {}),
                  ((kc, vc, slots, 128, ks, vs), dict(out_k=out[:4])), ((kc, vc, slots, 128, ks, vs), dict(out_k=out[:, :128])),
                  ((kc, vc, slots, 128, ks, vs), dict(out_k=out, out_v=out.float())),
                  ((kc.cpu(), vc, slots, 128, ks, vs), dict(out_k=out)), ((kc, vc, slots, 96, ks, vs), dict(out_k=out))):
        with pytest.raises(ValueError):
            qk.qknorm_paged_gather(*a, **kw)
    with pytest.raises(qk.QKNormError):
        qk.qknorm_paged_gather(kc, vc, slots, 128, ks, vs, out_k=out, out_v=out)
    for a, kw in (((kc, vc, slots, 128, ks, vs), dict(dtype=torch.float16)), ((kc, vc, slots, 128), {})):
        with pytest.raises(TypeError):
            qk.qknorm_paged_gather(*a, **kw)
