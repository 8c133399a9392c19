"""The lowest scale bytes of MXFP4 and MXFP8 caches, which another writer may have filled: a byte b
stands for 2^(b - 127), 0 for 2^-127. Read back and attended over, against the float64 oracle."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu
FORMATS = ["mxfp8", "mxfp4"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


def _values(fmt):
    return O.mxfp8_values if fmt == "mxfp8" else O.mxfp4_values


def _codes(r, fmt, shape, d, small=False, low=0):
    """Random codes, none of them NaN; small: of magnitudes up to 1; low: the least MXFP8 code."""
    if fmt == "mxfp4":
        c = r.integers(0, 3, (2,) + shape + (d // 2,)) + 8 * r.integers(0, 2, (2,) + shape + (d // 2,))
        return (c[0] | c[1] << 4).astype(np.uint8) if small else r.integers(0, 256, shape + (d // 2,), dtype=np.uint8)
    c = r.integers(low, 57 if small else 127, shape + (d,)) + 128 * r.integers(0, 2, shape + (d,))
    return c.astype(np.uint8)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,d,pad", [(2, 128, 0), (3, 96, 8), (1, 64, 3)])
def test_gather(fmt, dtype, heads, d, pad):
    """float32 holds every value exactly; bf16 those that are multiples of 2^-133, the others rounded."""
    print(f"[case] gather low scales {fmt} {dtype} {heads} {d} {pad}", flush=True)
    r = C.rng(d + pad)
    T, ps = 400, 16
    pages = T // ps
    codes = [_codes(r, fmt, (pages, heads, ps), d) for _ in range(2)]
    scales = [r.integers(0, 24, (pages, heads, ps, d // 32), dtype=np.uint8) for _ in range(2)]
    slots = r.permutation(pages * ps).astype(np.int64)
    out = [torch.full((T, heads * d + pad), 3.0, dtype=C.TORCH[dtype], device="cuda")[:, :heads * d] for _ in range(2)]
    dev = [torch.from_numpy(x).cuda() for x in codes + scales]
    qk.qknorm_paged_gather(dev[0], dev[1], C.dev(slots), d, dev[2], dev[3], *out)
    torch.cuda.synchronize()
    for i in range(2):
        want = _values(fmt)(codes[i][slots // ps, :, slots % ps], scales[i][slots // ps, :, slots % ps])
        got = C.host_values(out[i].contiguous()).reshape(T, heads, d)
        exact = want == np.ldexp(np.round(np.ldexp(want, 133)), -133) if dtype == "bf16" else np.ones(want.shape, bool)
        assert (exact & (scales[i][slots // ps, :, slots % ps].repeat(32, -1) == 0) & (want != 0)).any()
        assert np.array_equal(got[exact], want[exact])
        assert (np.abs(got - want)[~exact] <= 2.0 ** -134).all()        # half a step


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("d,hq,hk,n_q", [(64, 4, 2, 1), (128, 8, 2, 1), (256, 2, 1, 3), (64, 2, 1, 70), (128, 2, 1, 70),
                                         (128, 4, 1, 100), (256, 2, 1, 40)])
def test_attention(fmt, side, small, d, hq, hk, n_q):
    """Keys of the lowest scales against queries that bring their scores to about one, or values of
    the lowest scales; small: all of them below bf16's normal range. Codes of magnitudes from 2^-3
    on, whose values are multiples of 2^-133: bf16 holds them exactly. Tolerance as derived in
    test_attend_wide_gpu.py, with half a subnormal step for the result."""
    print(f"[case] attend low scales {fmt} {side} {small} {d} {n_q}", flush=True)
    r = C.rng(d + n_q)
    n, ps = 150, 16
    pages = -(-n // ps)
    codes = [_codes(r, fmt, (pages, hk, ps), d, small, 32) for _ in range(2)]
    top = 0 if small else 9 if fmt == "mxfp8" else 3                   # about the largest code, log2
    ordinary, low = 127 - top, r.integers(0, 3, (pages, hk, ps, d // 32), dtype=np.uint8)
    scales = [np.full((pages, hk, ps, d // 32), ordinary, np.uint8) for _ in range(2)]
    scales["kv".index(side)] = low
    # low keys: up to about 2^(top - 125)
    size = 2.0 ** (127 - top) / d ** 0.5 if side == "k" else 1.0
    q = C.to_type(np.clip(r.normal(size=(n_q, hq * d)), -3, 3) * size, "bf16")
    t = [torch.from_numpy(x).cuda() for x in codes + scales]
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens, cu = C.dev(np.array([n], np.int32)), C.dev(np.array([0, n_q], np.int32))
    if fmt == "mxfp8":
        out = qk.qknorm_paged_attend_wide(C.dev(q), t[0], t[1], table, lens, d, t[2], t[3], cu_q=cu, scale=1.0)
    else:
        out = qk.qknorm_paged_attend(C.dev(q), *t, table, lens, d, cu_q=cu, scale=1.0)
    torch.cuda.synchronize()
    K, V = (_values(fmt)(c, s).transpose(0, 2, 1, 3).reshape(-1, hk, d)[:n] for c, s in zip(codes, scales))
    qv = C.values(q).reshape(n_q, hq, d)
    want, mag, some = O.attend(qv, K, V, n_q, 1.0, True, 0)
    assert some.all()
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag + 2.0 ** -134
    # reading them as zeros would not pass: all tokens alike, or no result
    zeros = V[:n - n_q + 1].mean(0).repeat(hq // hk, 0) if side == "k" else 0.0
    assert (np.abs(want[0] - zeros) > bound[0]).mean() > 0.5
    C.close(C.host_values(out).reshape(want.shape), want, bound, "out")
