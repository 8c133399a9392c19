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
