"""Which stream the binding's own allocations belong to: decided on the host, with fakes of torch's stream calls."""
import contextlib

import pytest
import torch

import int8_kv_cache_quant_gb300 as k


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def current(monkeypatch):
    """The current stream's handle, as a list of the streams entered; 3 outside any of them."""
    entered = [3]

    @contextlib.contextmanager
    def enter(s):
        entered.append(s.cuda_stream)
        yield
        entered.pop()

    monkeypatch.setattr(k.kvq, "_stream", lambda s: entered[-1] if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    return entered


@pytest.mark.parametrize("stream,want", [(None, 3), (Stream(3), 3), (Stream(7), 7)])
@pytest.mark.parametrize("make", ["_empty", "_result"])
def test_allocations_are_made_on_the_stream_of_the_call(monkeypatch, current, make, stream, want):
    made = []
    empty = torch.empty

    def spy(*args, **kw):
        made.append(current[-1])
        return empty(*args, **kw)

    monkeypatch.setattr(torch, "empty", spy)
    t = getattr(k.kvq, make)((4, 2), torch.float32, "cpu", stream)
    assert made == [want] and current == [3]
    assert t.shape == (4, 2) and t.dtype is torch.float32
