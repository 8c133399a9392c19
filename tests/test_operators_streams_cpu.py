"""Which stream's memory the operators' Python calls take, without a GPU: torch's
stream functions are replaced by records of what is asked of them."""

import pytest
import torch

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
