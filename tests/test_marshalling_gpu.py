"""What the operators' marshalling refuses beyond the cases of the calls' own tests."""

import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from test_operators_run_gpu import D, EPS, _world

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


def test_flags_without_a_truth_value():
    """A flag that is neither true nor false is refused, and nothing is written."""
    w = _world(T=40, seed=21)
    before = w["x"].clone()
    neither = torch.zeros(2)
    with pytest.raises(TypeError, match="interleaved"):
        qk.qknorm_headwise_rope(w["q"], w["k"], w["gq"], w["gk"], EPS, D, w["table"], w["pos"], interleaved=neither)
    with pytest.raises(TypeError, match="causal"):
        qk.qknorm_paged_attend(w["aq"], w["kc"], w["vc"], w["ks"], w["vs"], w["bt"], w["lens"], D, cu_q=w["cu"],
                               causal=neither, out=w["o"])
    torch.cuda.synchronize()
    assert C.same_bits(w["x"], before) and not w["o"].any()


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("axis", [0, 1])
def test_cache_axes_of_length_one_carry_any_stride(axis, four):
    """One page, or one head: the stride of that axis says nothing, and K's may differ from V's."""
    T, ps, d = 16, 16, 64
    shape = [2, 3, ps]
    shape[axis] = 1
    heads = shape[1]
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, 2 * heads * d), generator=g, device="cuda").bfloat16()
    k, v = x[:, :heads * d], x[:, heads * d:]
    slots = torch.arange(T, device="cuda")

    def cache(n, dtype):
        """Packed, and the same with another stride (in odd steps) for the axis."""
        a, b = (torch.zeros(shape + [n], dtype=dtype, device="cuda") for _ in range(2))
        strides = list(b.stride())
        strides[axis] = 5 * strides[axis] + 3
        return a, b.as_strided(b.shape, strides)

    def pair():
        return (cache(d // 2, torch.uint8), cache(d // 32, torch.uint8)) if four else (cache(d, torch.bfloat16), None)

    (ka, va), sc = pair()
    want = [torch.zeros_like(t, memory_format=torch.contiguous_format) for t in (ka, ka)]
    ws = [torch.zeros_like(sc[0]) for _ in range(2)] if four else [None, None]
    qk.qknorm_paged_append(None, k, v, None, None, EPS, d, None, None, ka, va, slots, *(sc or (None, None)))
    qk.qknorm_paged_append(None, k, v, None, None, EPS, d, None, None, *want, slots, *ws)
    torch.cuda.synchronize()
    assert want[0].any() and C.same_bits(ka, want[0]) and C.same_bits(va, want[1])
    if four:
        assert C.same_bits(sc[0], ws[0]) and C.same_bits(sc[1], ws[1])
        table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        lens = torch.full((1,), T, dtype=torch.int32, device="cuda")
        o = [qk.qknorm_paged_attend(k[-1:], *c, *s, table, lens, d) for c, s in (((ka, va), sc), (want, ws))]
        assert C.same_bits(*o)
