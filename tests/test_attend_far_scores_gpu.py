"""qknorm_paged_attend with scores near the ends of float32's range, against the float64 oracle."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("d,n,n_q", [(64, 40, 1), (128, 3000, 1), (128, 70, 30), (256, 50, 1)])
def test_scores_of_the_largest_magnitude(d, n, n_q, sign):
    """Equal scores of +-2^127 weigh their tokens alike; scores 2^125 below them weigh nothing."""
    print(f"[case] far scores {d} {n} {n_q} {sign}", flush=True)
    r = C.rng(n + d)
    ps, hk, hq = 16, 1, 2
    pages = -(-n // ps)
    k = np.full((pages * ps, hk, d), 2.0 ** 60)
    low = r.random(n) < 0.4
    low[:n - n_q + 1] |= np.arange(n - n_q + 1) % 3 == 0
    low[0] = False
    k[:n][low] *= 1.5 if sign < 0 else 0.5
    v = r.normal(size=k.shape)
    if sign < 0:        # 1.5 * 2^127 fits float32, times log2 e it does not: such a score weighs nothing
        assert 1.5 * 2.0 ** 127 < 3.4e38 < 1.5 * 2.0 ** 127 * 1.4427
    codes, scales = zip(*(O.mxfp4_quantize(x.reshape(pages, ps, hk, d).transpose(0, 2, 1, 3))[:2] for x in (k, v)))
    q = C.to_type(np.full((n_q, hq * d), sign * 2.0 ** 67 / d), "bf16")
    t = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in codes + scales]
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out = qk.qknorm_paged_attend(C.dev(q), *t, table, C.dev(np.array([n], np.int32)), d,
                                 cu_q=C.dev(np.array([0, n_q], np.int32)), scale=1.0)
    torch.cuda.synchronize()
    K, V = (O.mxfp4_values(c, s).transpose(0, 2, 1, 3).reshape(-1, hk, d)[:n] for c, s in zip(codes, scales))
    want, mag, some = O.attend(C.values(q).reshape(n_q, hq, d), K, V, n_q, 1.0, True, 0)
    assert some.all()
    # scores are sums of equal powers of two, exact; the roundings of probabilities (1: none), result and sums
    C.close(C.host_values(out).reshape(want.shape), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag, "out")
