"""The helpers' workspace, on the host with the allocator replaced: whose memory
a buffer is."""
import contextlib

import pytest
import torch

import compensated_fp32_projection_amd as cf


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Buffer:
    """What torch.empty gives here: remembers the stream it was allocated under."""

    def __init__(self, nbytes, device, under):
        self.nbytes, self.device, self.under, self.used_on = nbytes, device, under, []

    def numel(self):
        return self.nbytes

    def data_ptr(self):
        return id(self)

    def record_stream(self, stream):
        self.used_on.append(stream)


@pytest.fixture
def allocator(monkeypatch):
    """Streams of the fake allocator: the current one, and what was allocated."""
    state = {"current": Stream(1), "made": []}

    @contextlib.contextmanager
    def under(stream):
        before, state["current"] = state["current"], stream or state["current"]
        yield
        state["current"] = before

    def empty(nbytes, dtype=None, device=None):
        state["made"].append(Buffer(nbytes, device, state["current"]))
        return state["made"][-1]

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state["current"])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(cf, "_default_ws", {})
    return state


def test_a_buffer_is_memory_of_the_stream_it_is_for(allocator):
    """Its first kernel runs on that stream: memory of another may still be in use there."""
    side, dev = Stream(2), torch.device("cuda", 0)
    ws = cf.Workspace()
    assert ws.get(100, dev, side).under is side and ws.buf.used_on == [side]
    assert ws.get(300, dev, side).under is side and ws.get(10, dev, side) is ws.buf
    assert [b.nbytes for b in allocator["made"]] == [100, 300]
    assert cf.Workspace().get(5, dev).under is allocator["current"]


def test_the_attention_helpers_take_it_there(allocator):
    side, dev = Stream(2), torch.device("cuda", 0)
    cf._scratch(64, dev, None, side)
    cf._scratch(64, dev, cf.Workspace(), side)
    cf._scratch(64, dev, None, None)
    assert [b.under.cuda_stream for b in allocator["made"]] == [2, 2, 1]
