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


def _prepare(w, **kw):
    attend = qk.prepare_paged_attend(w["aq"], w["kc"], w["vc"], w["ks"], w["vs"], w["bt"], w["lens"], D, cu_q=w["cu"],
                                     max_q=w["T"], **kw)
    grad = qk.prepare_headwise_rope_backward(w["yq"], w["yk"], w["q"], w["k"], w["gq"], w["gk"], EPS, D, w["table"],
                                             w["pos"])
    return attend, grad


def _decode_world(n):
    """One sequence of n tokens whose last is decoded: its cache is split over many blocks."""
    w = _world(T=n, seed=12)
    _everything(w)
    w["cu"] = None
    w["aq"] = w["aq"][-1:].clone()
    w["T"] = 1
    torch.cuda.synchronize()
    return w


def test_dropped_prepared_calls_keep_their_memory_while_they_run():
    """Prepared on the default stream, launched behind a long wait on another one and dropped:
    what the default stream allocates next is not the memory that the launch still uses."""
    w = _decode_world(9000)
    attend, grad = _prepare(w)
    want_o, want_g = attend().clone(), [t.clone() for t in grad()]
    torch.cuda.synchronize()
    assert attend._own[1].numel() > 0 and grad._own[-1].numel() > 0     # workspaces
    del attend, grad
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)           # some 10 ms
    attend, grad = _prepare(w)
    sizes = [t.numel() * t.element_size() for t in attend._own + grad._own]
    places = {t.data_ptr() for t in attend._own + grad._own}
    o, g = attend(stream=side), grad(stream=side.cuda_stream)
    with torch.cuda.stream(side):
        o, g = o.clone(), [t.clone() for t in g]
    del attend, grad
    new = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    assert not places & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    assert C.same_bits(o, want_o)
    for a, b in zip(g, want_g):
        assert C.same_bits(a, b)


def test_a_prepared_call_follows_lengths_and_pages_that_change_in_place():
    """A decode loop: seq_lens and block_table are rewritten between launches of one object, and
    between replays of a graph that holds it."""
    w = _decode_world(700)
    call = qk.prepare_paged_attend(w["aq"], w["kc"], w["vc"], w["ks"], w["vs"], w["bt"], w["lens"], D)

    def fresh():
        return qk.qknorm_paged_attend(w["aq"], w["kc"], w["vc"], w["ks"], w["vs"], w["bt"].clone(), w["lens"].clone(),
                                      D)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    torch.cuda.synchronize()
    g = torch.Generator(device="cuda").manual_seed(1)
    seen = []
    for n in (1, 16, 17, 333, 600, 700):
        w["lens"].fill_(n)
        w["bt"].copy_(torch.randperm(w["bt"].shape[1], generator=g, device="cuda").int()[None])
        want = fresh()
        got = call().clone()
        torch.cuda.synchronize()
        assert C.same_bits(got, want), n
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert C.same_bits(out, want), n
        seen.append(want)
    assert not any(C.same_bits(a, b) for a, b in zip(seen, seen[1:]))
