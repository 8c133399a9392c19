"""4-bit codes of keys whose sums, factors or products leave float32's normal range: they are
formed in float64, so codes and scales are still those of exact arithmetic."""

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


# row type, head width (96: the layout of pairs), rotated columns, interleaved
SHAPES = [("bf16", 128, 128, False), ("bf16", 128, 64, True), ("f32", 128, 128, False), ("f32", 256, 256, False),
          ("bf16", 96, 96, False), ("bf16", 512, 512, False)]


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("gammas", ["ordinary", "far"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_keys_far_from_one(shape, gammas, eps):
    dtype, d, rot, inter = shape
    print(f"[case] key codes {shape} {gammas} {eps}", flush=True)
    r = C.rng(d + rot)
    T, heads, ps = 130, 2, 16
    # rows from the subnormals to sums that overflow, each row of one magnitude
    scale = 2.0 ** np.linspace(-132, 123, T)[r.permutation(T)][:, None]
    host = C.to_type(np.clip(r.normal(size=(T, heads * d)) * scale, -3e38, 3e38), dtype)
    v = C.to_type(r.normal(size=(T, heads * d)), dtype)
    g = r.normal(1, 0.2, size=d)
    if gammas == "far":
        g = g * 2.0 ** r.integers(-90, 90, d)
    g = C.to_type(g, dtype)
    tab, pos = C.table(300, rot), r.integers(0, 300, T)
    pages = -(-T // ps)
    kc, vc = (torch.zeros((pages, heads, ps, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, heads, ps, d // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = np.arange(T, dtype=np.int64)
    qk.qknorm_paged_append(None, C.dev(host), C.dev(v), None, C.dev(g), eps, d, C.dev(tab), C.dev(pos), kc, vc,
                           C.dev(slots), ks, vs, inter)
    torch.cuda.synchronize()
    cos, sin = O.angles(tab, pos, rot)
    with np.errstate(all="ignore"):
        want = O.norm_rope(C.values(host), C.values(g), eps, d, 0, cos, sin, inter)
    codes, scales, _ = O.mxfp4_quantize(want)
    got_codes = kc.cpu().numpy()[slots // ps, :, slots % ps]
    got_scales = ks.cpu().numpy()[slots // ps, :, slots % ps]
    assert np.array_equal(got_scales, scales), f"{int((got_scales != scales).sum())} scales of {scales.size}"
    for a, b in ((got_codes & 15, codes & 15), (got_codes >> 4, codes >> 4)):
        assert ((a == b) | ((a & 7) + (b & 7) == 0)).all()      # the sign of a zero may differ
