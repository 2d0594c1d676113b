"""On which stream orthogonalize() takes the memory that it hands out. Streams
and launches are stood in for on the host: no kernel runs here."""
import contextlib

import pytest
import torch

import optimizer_step_layeradam_amd as la


class Stream:
    def __init__(self, name):
        self.cuda_stream = name


@pytest.fixture
def streams(monkeypatch):
    """The stream that is current at each allocation, in order; a stack of
    the current ones."""
    current = [Stream(1)]
    allocated = []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def recorded(make):
        def wrapped(*args, **kw):
            kw.pop("device", None)
            allocated.append(current[-1])
            return make(*args, **kw)
        return wrapped

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: current[-1])
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch, "empty_like", recorded(torch.empty_like))
    monkeypatch.setattr(la, "device_address", lambda t: t.data_ptr())
    monkeypatch.setattr(la, "_workspace_ptr", lambda t: t.data_ptr())
    monkeypatch.setattr(la, "orthogonalize_raw", lambda *args: launched.append(args[-1]))
    launched = []
    return current, allocated, launched


@pytest.mark.parametrize("turned", [False, True])
def test_default_outputs_belong_to_the_stream_that_writes_them(streams, turned):
    current, allocated, launched = streams
    x = [torch.zeros(5, 9), torch.zeros(2, 7, 3)]
    x = [t.mT for t in x] if turned else x
    s = Stream(2)
    la.orthogonalize(x, stream=s)
    assert launched == [2]
    assert len(allocated) == 3 and all(a is s for a in allocated)  # two outputs, the workspace
    allocated.clear()
    la.orthogonalize(x)
    assert launched == [2, 1]
    assert len(allocated) == 3 and all(a is current[0] for a in allocated)
