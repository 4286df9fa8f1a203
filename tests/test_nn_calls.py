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


def host_tensor(cbk):
    import numpy as np
    c = cbk.encode(np.arange(64 * 8, dtype=np.uint16).reshape(8, 64))
    return c.to("cpu")


@pytest.mark.parametrize("name", ["linear", "linear_dx", "ffn_gated", "ffn_gated_bwd", "xent", "xent_bwd"])
def test_tensors_that_ask_for_a_gradient_are_refused(name):
    """The results carry no graph, so a tensor whose gradient autograd is to compute is refused where autograd
    records, and taken under no_grad (the next check, for GPU tensors, is reached)."""
    import fly_decode_amd as cbk
    t = host_tensor(cbk)

    def call(wants):
        x, dy = (torch.zeros(3, n, dtype=torch.bfloat16) for n in (64, 8))
        labels, lse, dloss = torch.zeros(3, dtype=torch.int64), torch.zeros(3), torch.zeros(3)
        named = {"X": x, "dY": dy, "lse": lse, "dloss": dloss}
        named[wants].requires_grad_()
        return {"linear": lambda: cbk.linear(t, x), "linear_dx": lambda: cbk.linear_dx(t, dy),
                "ffn_gated": lambda: cbk.ffn_gated(t, t, x), "ffn_gated_bwd": lambda: cbk.ffn_gated_bwd(t, t, x, dy),
                "xent": lambda: cbk.xent(t, x, labels),
                "xent_bwd": lambda: cbk.xent_bwd(t, x, labels, lse, dloss)}[name]()

    takes = {"linear": ["X"], "linear_dx": ["dY"], "ffn_gated": ["X"], "ffn_gated_bwd": ["X", "dY"], "xent": ["X"],
             "xent_bwd": ["X", "lse", "dloss"]}[name]
    for wants in takes:
        with pytest.raises(ValueError, match="no_grad"):
            call(wants)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            call(wants)


def test_the_stride_of_a_single_row_means_nothing():
    """One row, or none, of a view whose row stride is past the limit on leading dimensions, or below the width."""
    import fly_decode_amd as cbk
    x = torch.zeros(64, dtype=torch.bfloat16)
    for stride in (0, 1, 64, 1 << 33):
        for rows in (0, 1):
            _, ld = cbk._tokens(x.as_strided((rows, 64), (stride, 1)), 64, "X")
            assert 64 <= ld < 1 << 32
    with pytest.raises(ValueError, match="overlap"):
        cbk._tokens(x.as_strided((2, 32), (16, 1)), 32, "X")
