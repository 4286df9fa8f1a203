"""CPU tests of what the binding of the operators in include/cbk_nn.h does around a call: where its
allocations come from and what it refuses (torch's allocator and streams are replaced by records of
their use; no GPU is needed)."""
import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

DEVICE = torch.device("cuda", 0)


class Block:
    """An allocation: the stream whose pool it came from, and the streams it was recorded on."""

    def __init__(self, pool):
        self.pool, self.recorded = pool, []

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def streams(monkeypatch):
    """(the current stream, another one); torch.empty gives a Block of the stream that is current then."""
    current = SimpleNamespace(device=DEVICE, cuda_stream=16)
    other = SimpleNamespace(device=DEVICE, cuda_stream=32)
    now = [current]

    @contextlib.contextmanager
    def switch(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Block(now[-1]))
    return current, other


def call_on(stream):
    import fly_decode_amd
    return fly_decode_amd._Call(SimpleNamespace(device=DEVICE), stream)


def test_allocations_come_from_the_stream_that_the_call_runs_on(streams):
    """A block of another stream's pool may have been freed with that stream's work on it still to run, which
    the call's stream does not wait for."""
    current, other = streams
    block = call_on(None).empty((4,), torch.uint8)
    assert block.pool is current
    block = call_on(current).empty((4,), torch.uint8)
    assert block.pool is current
    block = call_on(other).empty((4,), torch.uint8)
    assert block.pool is other


def test_outputs_are_kept_for_the_current_stream_too(streams):
    """The caller goes on with an output on its current stream, whose work on it the allocator has to wait
    for when the output is freed."""
    current, other = streams
    assert call_on(other).empty((4,), torch.uint8).recorded == [current]
    assert call_on(None).empty((4,), torch.uint8).recorded == []


def test_a_stream_of_another_device_is_refused(streams):
    elsewhere = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=48)
    with pytest.raises(ValueError, match="stream"):
        call_on(elsewhere)
