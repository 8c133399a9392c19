"""Which stream's memory the operators' Python calls take, without a GPU: torch's
stream functions are replaced by records of what is asked of them."""

import os

import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
from layerwise_qk_norm_qknorm_amd import operators


class Stream:
    def __init__(self, name, handle):
        self.name, self.cuda_stream = name, handle


@pytest.fixture
def streams(monkeypatch):
    """torch.cuda as far as the calls use it; the context returned is the stream it was given."""
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Stream("external", h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream("default", 0))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)


def test_memory_for_a_stream_handle(streams):
    dev = torch.device("cuda", 0)
    assert operators._at(None, dev) is None                 # no change of stream
    own = Stream("own", 77)
    assert operators._at(own, dev) is own
    s = operators._at(99, dev)
    assert (s.name, s.cuda_stream) == ("external", 99)
    assert operators._at(0, dev).name == "default"          # the default stream, not a new one


class Memory:
    def __init__(self):
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append((stream.name, stream.cuda_stream))


def test_a_prepared_call_records_the_streams_it_runs_on(streams, monkeypatch):
    """What was allocated for a prepared call is recorded on every other stream that the call is
    launched on, so that the allocator waits for them before it hands the memory out again."""
    now = {"stream": 5}
    launched = []

    class Native:
        @staticmethod
        def launch(call, s):
            launched.append(s)
            return 0

    monkeypatch.setattr(operators, "_native", lambda: Native)
    monkeypatch.setattr(operators, "_raw_stream", lambda dev: now["stream"])
    monkeypatch.setattr(operators, "_current_device", lambda: 0)
    memory = Memory()
    call = operators._OperatorCall(object(), 0, "result", (memory,))
    assert call() == "result" and memory.recorded == []        # the stream it was allocated on
    call(stream=5)
    assert memory.recorded == []
    call(stream=Stream("own", 77))
    call(stream=Stream("own", 77))                              # once a stream
    assert memory.recorded == [("own", 77)]
    now["stream"] = 31                                          # another current stream
    call()
    call(stream=0)
    assert memory.recorded[1:] == [("external", 31), ("default", 0)]
    assert launched == [5, 5, 77, 77, 31, 0]
    operators._OperatorCall(object(), 0, None)(stream=77)      # nothing of its own: nothing to record


@pytest.mark.skipif(not os.path.exists(qk.library_path()),
                    reason="libqknorm.so not built (run __graft_entry__.build())")
def test_prepared_calls_refuse_tensors_that_are_not_on_a_gpu():
    q, k = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16)
    g = torch.ones(128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        qk.prepare_headwise_rope_backward(q, k, q, k, g, g, 1e-6, 128, None, None)
    cache = [torch.zeros(2, 1, 16, n, dtype=torch.uint8) for n in (64, 64, 4, 4)]
    one = torch.ones(4, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        qk.prepare_paged_attend(q, *cache, one, one[:, 0].contiguous(), 128)
