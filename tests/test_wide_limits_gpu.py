"""Calls over wide caches at their limits: more sequences than a wave orders, row tiles that a block
takes in turn, capped grids, pages, tokens and rows past 32-bit offsets, equal results of equal
calls."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from test_attend_wide_gpu import FORMATS, Case
from wide_cap_cases import CASES, run

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("less than 64 GiB of device memory free")
    qk.load_library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [63, 64, 65, 90])
@pytest.mark.parametrize("d,group", [(128, 1), (128, 5), (64, 4), (256, 2)])
def test_sequences_around_what_a_wave_orders(B, d, group, fmt):
    """Sequences of no rows, one row and many, and of no tokens, among them."""
    r = C.rng(B + d)
    n_q = [int(n) for n in r.integers(0, 60, B)]
    lens = [n + int(r.integers(0, 150)) for n in n_q]
    n_q[0], lens[0] = 1, 1
    n_q[B // 2], lens[B // 2] = 0, 400
    n_q[B - 1], lens[B - 1] = 40, 0
    n_q[B - 2], lens[B - 2] = 70, 300
    c = Case(fmt, 100 + B, d, 2 * group, 2, lens, n_q, 16)
    c.check(c.run(max_q=70, max_len=512))
    c.check(c.run())                              # bounds from the shapes: more blocks than rows


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [2, 70])
@pytest.mark.parametrize("d,group,bound", [(128, 4, 33), (128, 4, 9), (64, 4, 20), (256, 1, 40)])
def test_blocks_take_rows_in_turn(B, d, group, bound, fmt):
    """max_q names fewer rows than the longest sequence has, so that blocks loop over its rows."""
    r = C.rng(B + d + group)
    n_q = [int(n) for n in r.integers(0, 12, B)]
    n_q[1] = 310
    lens = [n + int(r.integers(0, 90)) for n in n_q]
    c = Case(fmt, 7, d, group, 1, lens, n_q, 32)
    c.check(c.run(max_q=bound, max_len=400))
    c.check(c.run(max_q=bound, max_len=400, window=37), window=37)


@pytest.mark.parametrize("fmt", FORMATS)
def test_equal_calls_give_equal_bits(fmt):
    for n_q, lens in (([1, 1], [5000, 300]), ([300, 20], [1300, 900])):
        c = Case(fmt, 11, 128, 8, 2, lens, n_q, 64)
        a = c.run()
        for _ in range(3):
            assert C.same_bits(a, c.run())


@pytest.fixture(scope="module")
def capped(tmp_path_factory):
    assert "QKNORM_MAX_GRID" not in os.environ, "the uncapped calls need the variable unset"
    out = str(tmp_path_factory.mktemp("cap") / "capped.npz")
    res = subprocess.run([sys.executable, "-u", os.path.join(HERE, "wide_cap_cases.py"), out],
                         env=dict(os.environ, QKNORM_MAX_GRID="7"), capture_output=True, text=True, timeout=200)
    print(res.stdout[-2000:], res.stderr[-2000:], flush=True)
    assert res.returncode == 0, f"child process failed ({res.returncode})"
    with np.load(out) as d:
        return {k: d[k] for k in d.files}


@pytest.mark.parametrize("i", range(len(CASES)), ids=lambda i: "-".join(str(x) for x in CASES[i]))
def test_capped_grids_give_the_same_bits(i, capped):
    print(f"[case] cap {CASES[i]}", flush=True)
    for n, a in enumerate(run(CASES[i])):
        assert np.array_equal(a, capped[f"{i}_{n}"]), n


def _bytes_far(shape, strides, fmt):
    """A cache array of these strides (elements), and one in one piece."""
    t = torch.uint8 if fmt == "mxfp8" else torch.bfloat16
    room = torch.empty(sum((n - 1) * s for n, s in zip(shape, strides)) + 1, dtype=t, device="cuda")
    far = room.as_strided(shape, strides)
    far.zero_()
    return far, torch.zeros(shape, dtype=t, device="cuda")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,n_q", [(6, 1), (700, 700), (700, 16), (700, 30), (700, 1)])
@pytest.mark.parametrize("layout", ["pages", "tokens", "heads"])
def test_caches_past_32_bits(layout, T, n_q, fmt):
    """Pages 2^30 or heads 2^31 elements and a bit apart, or tokens nearly 2^28 bytes, the most that
    attention takes: appending to such a cache, reading it back and attending over it give the bits
    of a cache in one piece."""
    print(f"[case] far: {layout} {T} {n_q} {fmt}", flush=True)
    d, hq, hk, ps = 128, 10, 2, 64
    if layout == "tokens":
        ps = 32
    pages = -(-T // ps) + 1
    apart = 1024
    strides = {"pages": ((1 << 30) + apart, ps * d, d, 1),
               "tokens": (hk * d, d, (1 << (28 if fmt == "mxfp8" else 27)) - apart, 1),
               "heads": (ps * d, (1 << 31) + apart, d, 1)}[layout]
    shape = (pages, hk, ps, d)
    caches = [_bytes_far(shape, strides, fmt) for _ in range(2)]
    scales = [[torch.zeros((pages, hk, ps, d // 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
              if fmt == "mxfp8" else [None, None] for _ in range(2)]
    x = torch.from_numpy(C.rng(5).normal(size=(T, (hq + 2 * hk) * d))).to(torch.bfloat16).cuda()
    q, k, v = x.split([hq * d, hk * d, hk * d], 1)
    td = C.dev(C.table(1024, d))
    pos = torch.stack([torch.arange(T, device="cuda"), torch.arange(T, device="cuda") // 7])
    names = qk.rope_axes((30, 34))
    table = torch.from_numpy(C.rng(6).permutation(pages).astype(np.int32)[None]).cuda()
    slots = table[0].long()[pos[0] // ps] * ps + pos[0] % ps
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, n_q], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    outs = []
    for i in range(2):
        ck, cv = caches[0][i], caches[1][i]
        oq = torch.empty((T, hq * d), dtype=torch.bfloat16, device="cuda")
        qk.qknorm_paged_append_axes(q, k, v, gamma, gamma, EPS, d, td, pos, names, ck, cv, slots, *scales[i], out_q=oq)
        rows = qk.qknorm_paged_gather(ck, cv, slots, d, *scales[i])
        o = qk.qknorm_paged_attend_wide(oq[T - n_q:], ck, cv, table, lens, d, *scales[i], cu_q=cu, max_q=n_q, max_len=T)
        outs.append((oq, *rows, o, *(s for s in scales[i] if s is not None)))
    torch.cuda.synchronize()
    for f, n in caches:
        assert C.same_bits(f, n)
    for a, b in zip(*outs):
        assert C.same_bits(a, b)
    assert outs[0][3].float().abs().max() > 0


def test_rows_read_back_past_32_bits():
    """Rows 2^30 elements and a bit apart, and rows that no slot fills stay as they were."""
    d, heads, ps, pages, T, ld = 128, 2, 16, 9, 6, (1 << 30) + 1024
    cache = [torch.randn((pages, heads, ps, d), device="cuda").bfloat16() for _ in range(2)]
    slots = torch.tensor([140, 3, -1, 3, 80, 0], device="cuda")
    room = torch.full(((T - 1) * ld + heads * d,), 3.0, dtype=torch.bfloat16, device="cuda")
    far = room.as_strided((T, heads * d), (ld, 1))
    _, v = qk.qknorm_paged_gather(*cache, slots, d, out_k=far)
    assert v is None
    torch.cuda.synchronize()
    for t, s in enumerate(slots.tolist()):
        want = cache[0][s // ps, :, s % ps].reshape(-1) if s >= 0 else torch.full((heads * d,), 3.0, device="cuda").bfloat16()
        assert C.same_bits(far[t], want), t


@pytest.mark.parametrize("T", [2049, 9001])
@pytest.mark.parametrize("d", [80, 96, 192])
def test_waves_of_several_tokens(d, T):
    """More tokens than the chip holds waves of: the bits of calls of 300 tokens, which it does hold."""
    hq, hk, ps = 24, 5, 16
    r = C.rng(T)
    x = torch.randn((T, (hq + 2 * hk) * d), generator=torch.Generator(device="cuda").manual_seed(d), device="cuda").bfloat16()
    q, k, v = x.split([hq * d, hk * d, hk * d], 1)
    gamma = [torch.from_numpy(r.normal(1, 0.2, d)).bfloat16().cuda() for _ in range(2)]
    td, pos = C.dev(C.table(512, d)), C.dev(r.integers(0, 512, (3, T)))
    names = qk.rope_axes((d // 2 - 20, 10, 10))
    slots = C.dev(r.permutation(T + 50)[:T].astype(np.int64))
    pages = -(-(T + 50) // ps)

    def run(step):
        oq, ok = torch.empty((T, hq * d), dtype=x.dtype, device="cuda"), torch.empty((T, hk * d), dtype=x.dtype, device="cuda")
        out = [oq, ok]
        for t in range(0, T, step):
            s = slice(t, min(T, t + step))
            qk.qknorm_headwise_rope_axes(q[s], k[s], *gamma, EPS, d, td, pos[:, s], names, out_q=oq[s], out_k=ok[s])
        if d % 32 == 0:
            cache = [torch.zeros((pages, hk, ps, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
            scales = [torch.zeros((pages, hk, ps, d // 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
            aq = torch.empty_like(oq)
            for t in range(0, T, step):
                s = slice(t, min(T, t + step))
                qk.qknorm_paged_append(q[s], k[s], v[s], *gamma, EPS, d, td, pos[0, s], *cache, slots[s], *scales,
                                       out_q=aq[s])
            out += cache + scales + [aq]
        torch.cuda.synchronize()
        return out

    for a, b in zip(run(T), run(300)):
        assert C.same_bits(a, b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_q", [25, 26, 51, 52, 64, 76, 77])
def test_rows_around_whole_blocks(n_q, fmt):
    """Blocks of 128 and 256 rows: 125 to 385 rows of a sequence."""
    c = Case(fmt, n_q, 128, 10, 2, [700, n_q, 97], [n_q, n_q, 3], 32)
    for causal, window in ((True, 0), (False, 0), (True, 50)):
        c.check(c.run(causal=causal, window=window, max_q=n_q, max_len=700), causal=causal, window=window)
