"""qknorm_paged_attend_wide with scores far from zero, against the float64 oracle: every row is
compared, whatever its scores."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu
FORMATS = ["rows", "mxfp8"]
SHAPES = [(64, 40, 1), (128, 3000, 1), (128, 70, 30), (256, 50, 1), (64, 200, 90), (128, 300, 200), (256, 120, 100)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


def _run(fmt, q, k, v, d, n_q, causal=True):
    """One sequence of k, v [n, heads, d] in pages of 16; (out, K, V as the cache holds them)."""
    n, hk = k.shape[:2]
    ps, pages = 16, -(-k.shape[0] // 16)
    pad = [np.concatenate((x, np.zeros((pages * ps - n, hk, d)))).reshape(pages, ps, hk, d).transpose(0, 2, 1, 3)
           for x in (k, v)]
    if fmt == "rows":
        host = [C.to_type(np.ascontiguousarray(x), "bf16") for x in pad]
        cache, scales = [C.dev(x) for x in host], {}
        held = [C.values(x) for x in host]
    else:
        codes, s, held = zip(*(O.mxfp8_quantize(x) for x in pad))
        cache = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in codes]
        s = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in s]
        scales = dict(k_scales=s[0], v_scales=s[1])
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = qk.qknorm_paged_attend_wide(C.dev(q), *cache, table, C.dev(np.array([n], np.int32)), d,
                                      cu_q=C.dev(np.array([0, n_q], np.int32)), scale=1.0, causal=causal, **scales)
    torch.cuda.synchronize()
    return (C.host_values(out),) + tuple(x.transpose(0, 2, 1, 3).reshape(-1, hk, d)[:n] for x in held)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("d,n,n_q", SHAPES)
def test_scores_of_the_largest_magnitude(fmt, d, n, n_q, sign):
    """Equal scores of +-2^127 weigh their tokens alike; scores 2^126 below them weigh nothing.
    Scores are sums of equal powers of two, exact in float32; the tolerance counts the roundings of
    probabilities (none: they are 1 or 0), the result and the sums."""
    print(f"[case] far scores wide {fmt} {d} {n} {n_q} {sign}", flush=True)
    r = C.rng(n + d)
    k = np.full((n, 1, d), 2.0 ** 60)
    low = r.random(n) < 0.4
    low[:n - n_q + 1] |= np.arange(n - n_q + 1) % 3 == 0
    low[0] = False
    k[low] *= 1.5 if sign < 0 else 0.5
    q = C.to_type(np.full((n_q, 2 * d), sign * 2.0 ** 67 / d), "bf16")
    got, K, V = _run(fmt, q, k, r.normal(size=k.shape), d, n_q)
    want, mag, some = O.attend(C.values(q).reshape(n_q, 2, d), K, V, n_q, 1.0, True, 0)
    assert some.all()
    C.close(got.reshape(want.shape), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag, "out")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("d,n,n_q", SHAPES)
def test_scores_that_climb_or_fall_along_the_cache(fmt, d, n, n_q, rising):
    """Token t's score is 32 t above -16 n, or below 16 n: the running maximum moves with every
    tile, or never again. One token carries all of a row (the next weighs e^-32): the last it sees,
    or the first. Scores are sums of four products of integers, exact."""
    print(f"[case] climbing scores wide {fmt} {d} {n} {n_q} {rising}", flush=True)
    r = C.rng(n * d)
    t = np.arange(n)
    step = (t if rising else n - 1 - t) - n // 2
    k = np.zeros((n, 1, d))
    # in base 8: digits that MXFP8 and bf16 hold exactly, the first of them negative for some
    parts = ((step // 512, 512.0), (step % 512 // 64, 64.0), (step % 64 // 8, 8.0), (step % 8, 1.0))
    q = np.zeros((n_q, 2, d))
    for (x, unit), c in zip(parts, (0, 1, 33, d - 1)):
        k[:, 0, c] = x
        q[:, :, c] = 32.0 * unit
    got, K, V = _run(fmt, C.to_type(q.reshape(n_q, -1), "bf16"), k, r.normal(size=k.shape), d, n_q)
    assert np.array_equal(K, k)
    want, mag, some = O.attend(q, K, V, n_q, 1.0, True, 0)
    assert some.all()
    C.close(got.reshape(want.shape), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag, "out")
