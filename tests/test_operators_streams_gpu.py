"""Streams and the memory that the operators' Python calls take for themselves."""

import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from layerwise_qk_norm_qknorm_amd import operators
from test_operators_run_gpu import D, EPS, _everything, _world

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


def test_handle_zero_is_the_default_stream():
    """Memory that a call with stream=0 allocates belongs to the default stream."""
    dev = torch.device("cuda", torch.cuda.current_device())
    with operators._at(0, dev):
        assert torch.cuda.current_stream().cuda_stream == 0
    side = torch.cuda.Stream()
    with operators._at(side.cuda_stream, dev):
        assert torch.cuda.current_stream().cuda_stream == side.cuda_stream
    w = _world(seed=11)
    _everything(w)
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.default_stream()):
        o = qk.qknorm_paged_attend(w["aq"], w["kc"], w["vc"], w["ks"], w["vs"], w["bt"], w["lens"], D, cu_q=w["cu"],
                                   max_q=w["T"], stream=stream)
        g = qk.qknorm_headwise_rope_backward(w["yq"], w["yk"], w["q"], w["k"], w["gq"], w["gk"], EPS, D, w["table"],
                                             w["pos"], stream=stream)
        torch.cuda.synchronize()
        assert C.same_bits(o, w["o"])
        assert C.same_bits(g[0], w["dq"]) and C.same_bits(g[2], w["dgq"])
