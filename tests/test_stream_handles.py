"""The stream handle that the serving calls run on is the caller's, 0 (the default stream) among them; checked without
a device against stand-ins for torch's stream objects."""
import contextlib

import pytest
import torch

from post_weight_quantization_hessian_b200 import slim

POOL = 0x5000   # what torch returns for an external stream of handle 0: a stream of its own pool


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def entered(monkeypatch):
    streams = []

    @contextlib.contextmanager
    def guard(s):
        streams.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", guard)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: FakeStream(h or POOL))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    return streams


@pytest.mark.parametrize("given, handle", [(0, 0), (0x1230, 0x1230), (FakeStream(0), 0), (FakeStream(0x77), 0x77)])
def test_the_call_runs_on_the_given_handle(entered, given, handle):
    with slim._on(torch.device("cuda", 0), given) as raw:
        assert raw == handle
    assert [s.cuda_stream for s in entered] == [handle]
