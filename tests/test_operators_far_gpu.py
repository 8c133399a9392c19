"""Sizes past 32 bits and launches past one grid: rows, pages and caches whose
elements lie beyond 2^32 bytes of their base, token counts that a launch goes
through in several passes, and windows narrower than the part of the cache one
block takes."""

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
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("less than 48 GiB of device memory free")
    qk.load_library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _table(n, rot):
    t = C.table(n, rot)
    return t, C.dev(t)


def test_more_tokens_than_one_grid_of_waves():
    """2^22 blocks of four waves take 2^23 tokens of these two heads: the rest loop."""
    print("[case] far: tokens", flush=True)
    T, d = (1 << 23) * 2 + 77, 64
    host, td = _table(512, d)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((T, 2 * d), generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(T, device="cuda") % 512
    gamma = torch.full((d,), 1.25, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    qk.qknorm_headwise_rope(x[:, :d], x[:, d:], gamma, gamma, EPS, d, td, pos, out_q=out[:, :d], out_k=out[:, d:])
    torch.cuda.synchronize()
    step = 1 << 20
    part = torch.empty((step, 2 * d), dtype=torch.bfloat16, device="cuda")
    for t in range(0, T, step):     # the same rows in calls of one pass each
        n = min(step, T - t)
        qk.qknorm_headwise_rope(x[t:t + n, :d], x[t:t + n, d:], gamma, gamma, EPS, d, td, pos[t:t + n],
                                out_q=part[:n, :d], out_k=part[:n, d:])
        assert C.same_bits(out[t:t + n], part[:n]), t
    for t in (0, (1 << 23) - 8, T - 16):
        rows = x[t:t + 16, :d]
        p = pos[t:t + 16].cpu().numpy()
        z = O.norm_rope(C.host_values(rows), np.full(d, 1.25), EPS, d, 0, None, None, False)
        cos, sin = (host[p][:, i * d // 2:(i + 1) * d // 2].astype(np.float64) for i in (0, 1))
        C.close(C.host_values(out[t:t + 16, :d]).reshape(z.shape), O.rotate(z, cos, sin, False),
                C.rope_bound(z, cos, sin, False, "bf16"), f"rows {t}")


@pytest.mark.parametrize("d", [128, 80])
def test_rows_far_apart(d):
    """Rows 2^31 + 2^20 bytes apart: the third begins past 2^32."""
    print(f"[case] far: rows {d}", flush=True)
    T, hq, hk, ld = 4, 4, 2, (1 << 30) + (1 << 19)
    room = torch.empty((T - 1) * ld + (hq + hk) * d, dtype=torch.bfloat16, device="cuda")
    far = room.as_strided((T, (hq + hk) * d), (ld, 1))
    near = torch.from_numpy(C.rng(3).normal(size=far.shape)).to(torch.bfloat16).cuda()
    dy = torch.from_numpy(C.rng(4).normal(size=far.shape)).to(torch.bfloat16).cuda()
    _, td = _table(16, d)
    pos = torch.tensor([3, 0, 15, 7], device="cuda")
    gamma = torch.full((d,), 0.75, dtype=torch.bfloat16, device="cuda")
    split = lambda t: (t[:, :hq * d], t[:, hq * d:])
    far.copy_(near)
    qk.qknorm_headwise_rope(*split(far), gamma, gamma, EPS, d, td, pos)
    a = torch.cat([t.clone() for t in split(far)], 1)
    b = near.clone()
    qk.qknorm_headwise_rope(*split(b), gamma, gamma, EPS, d, td, pos)
    torch.cuda.synchronize()
    assert C.same_bits(a, b)
    far.copy_(near)
    g1 = qk.qknorm_headwise_rope_backward(*split(dy), *split(far), gamma, gamma, EPS, d, td, pos)
    g2 = qk.qknorm_headwise_rope_backward(*split(dy), *split(near), gamma, gamma, EPS, d, td, pos)
    torch.cuda.synchronize()
    for x, y in zip(g1, g2):
        assert C.same_bits(x, y)


@pytest.mark.parametrize("T", [6, 700])
def test_pages_far_apart(T):
    """A cache whose pages lie 2^30 + 2^10 bytes apart (a slice of a larger pool): appending
    to it and attending over it give the bits of a cache in one piece."""
    print(f"[case] far: pages {T}", flush=True)
    d, hq, hk, ps, pages = 128, 10, 2, 64, 12
    stride = (1 << 30) + 1024
    shape = (pages, hk, ps)
    room = [torch.empty((pages - 1) * stride + hk * ps * d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    far = [r.as_strided(shape + (d // 2,), (stride, ps * d // 2, d // 2, 1)) for r in room]
    near = [torch.zeros(shape + (d // 2,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [[torch.zeros(shape + (d // 32,), dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]
    for f in far:
        f.zero_()
    x = torch.from_numpy(C.rng(5).normal(size=(T, (hq + 2 * hk) * d))).to(torch.bfloat16).cuda()
    q, k, v = x.split([hq * d, hk * d, hk * d], 1)
    _, td = _table(1024, d)
    pos = torch.arange(T, device="cuda")
    table = torch.from_numpy(C.rng(6).permutation(pages).astype(np.int32)[None]).cuda()
    slots = table[0].long()[pos // ps] * ps + pos % ps
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    outs = []
    for c, s in ((far, scales[0]), (near, scales[1])):
        oq = torch.empty((T, hq * d), dtype=torch.bfloat16, device="cuda")
        qk.qknorm_paged_append(q, k, v, gamma, gamma, EPS, d, td, pos, c[0], c[1], slots, s[0], s[1], out_q=oq)
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        lens = torch.tensor([T], dtype=torch.int32, device="cuda")
        outs.append(qk.qknorm_paged_attend(oq, c[0], c[1], s[0], s[1], table, lens, d, cu_q=cu, max_q=T, max_len=T))
    torch.cuda.synchronize()
    assert all(C.same_bits(f, n) for f, n in zip(far, near))
    assert all(C.same_bits(f, n) for f, n in zip(*scales))
    assert C.same_bits(*outs) and bool(outs[0].isfinite().all())


@pytest.mark.parametrize("window", [1, 255, 300, 1500, 4000])
@pytest.mark.parametrize("max_len", [None, 64])
def test_windows_of_a_long_cache(window, max_len):
    """The cache is split over the window, not over the sequence; with a bound on the
    lengths that is too low as well."""
    print(f"[case] far: window {window} {max_len}", flush=True)
    r = C.rng(window)
    d, hq, hk, ps, n_q = 64, 6, 2, 16, [1, 3, 1]
    lens = [5000, 3333, 20]
    pages = sum(-(-n // ps) for n in lens)
    codes, scales = zip(*(O.mxfp4_quantize(r.normal(size=(pages, hk, ps, d)))[:2] for _ in range(2)))
    width = -(-max(lens) // ps)
    table = np.full((len(lens), width), -1, np.int32)
    ids, at = r.permutation(pages), 0
    for b, n in enumerate(lens):
        m = -(-n // ps)
        table[b, :m] = ids[at:at + m]
        at += m
    q = C.to_type(r.normal(size=(sum(n_q), hq * d)) * 1.5, "bf16")
    cu = np.concatenate(([0], np.cumsum(n_q))).astype(np.int32)
    t = [torch.from_numpy(x.copy()).cuda() for x in (codes[0], codes[1], scales[0], scales[1])]
    out = qk.qknorm_paged_attend(C.dev(q), *t, C.dev(table), C.dev(np.array(lens, np.int32)), d, cu_q=C.dev(cu),
                                 max_q=max(n_q), max_len=max_len or max(lens), window=window)
    torch.cuda.synchronize()
    got = C.host_values(out).reshape(-1, hq, d)
    qv = C.values(q).reshape(-1, hq, d)
    for b, n in enumerate(lens):
        m = -(-n // ps)
        k, v = (O.mxfp4_values(codes[i][table[b, :m]], scales[i][table[b, :m]]).transpose(0, 2, 1, 3)
                .reshape(-1, hk, d)[:n] for i in (0, 1))
        for i in range(n_q[b]):
            p = n - n_q[b] + i
            lo = max(p - window + 1, 0)
            for h in range(hq):
                s = k[lo:p + 1, h // 3] @ qv[cu[b] + i, h] / 8
                w = np.exp(s - s.max())
                w /= w.sum()
                want, mag = w @ v[lo:p + 1, h // 3], w @ np.abs(v[lo:p + 1, h // 3])
                # the roundings of the result and of the probabilities, and float32 sums
                C.close(got[cu[b] + i, h], want, 2.0 ** -8 * np.abs(want) + 2 * 2.0 ** -8 * mag, f"{b} {i} {h}")
