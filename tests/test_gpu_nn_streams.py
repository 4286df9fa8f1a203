"""GPU tests of calls of the operators in include/cbk_nn.h on a stream that the caller names, with nothing
but the inputs ordered before them: other work is still to run on the current stream."""
import pytest

import nn_reference as ref
from test_gpu_nn import acts, compress, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


def delay(torch, big):
    """Some milliseconds of work for the current stream."""
    for _ in range(20):
        big.mul_(1.0)


@pytest.mark.parametrize("T,rows,cols", [(1, 500, 256), (40, 500, 256), (400, 500, 192)])
def test_a_call_on_another_stream_beside_pending_work(env, T, rows, cols):
    """A call on the current stream that waits behind other work has returned its workspace; a call of the
    same kind on another stream runs meanwhile.  Each gives what it gives alone."""
    torch, cbk = env
    w = [weights(torch, rows, cols, 1500, 111 + i, 0.2) for i in range(2)]
    a, b = (compress(cbk, t) for t in w)
    x = [acts(torch, T, cols, 113 + i) for i in range(2)]
    xd = [t.cuda() for t in x]
    big = torch.ones(1 << 28, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ys, zs = [], []
    for _ in range(3):
        delay(torch, big)
        ys.append(cbk.linear(a, xd[0]))
        zs.append(cbk.linear(b, xd[1], stream=s))
    torch.cuda.synchronize()
    for y, z in zip(ys, zs):
        ref.assert_within(y, *ref.linear(x[0], w[0]), "current stream")
        ref.assert_within(z, *ref.linear(x[1], w[1]), "other stream")


@pytest.mark.parametrize("T", [1, 40])
def test_an_output_is_kept_while_the_current_stream_reads_it(env, T):
    """An output of a call on another stream, used on the current one and freed with that use still to run:
    the next call on the other stream does not write over it."""
    torch, cbk = env
    rows, cols = 500, 256
    w = weights(torch, rows, cols, 1500, 115, 0.2)
    a = compress(cbk, w)
    x = [acts(torch, T, cols, 116 + i) for i in range(2)]
    xd = [t.cuda() for t in x]
    big = torch.ones(1 << 28, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = cbk.linear(a, xd[0], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    delay(torch, big)
    copy = y.clone()
    del y
    later = [cbk.linear(a, xd[1], stream=s) for _ in range(4)]
    torch.cuda.synchronize()
    ref.assert_within(copy, *ref.linear(x[0], w), "the first output")
    for z in later:
        ref.assert_within(z, *ref.linear(x[1], w), "the later ones")
