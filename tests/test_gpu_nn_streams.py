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


@pytest.mark.parametrize("T", [1, 40, 400])
def test_a_captured_call_on_a_forked_stream(env, T):
    """Inside a capture, a call on a stream that was forked from the captured one, its outputs used behind the
    join: every replay against the eager call's bits, with eager calls between."""
    torch, cbk = env
    rows, cols = 320, 192
    wg, wu = (weights(torch, rows, cols, 1500, 118 + i, 0.2) for i in range(2))
    a, b = compress(cbk, wg), compress(cbk, wu)
    X, dH = (torch.empty(T, n, dtype=torch.bfloat16, device="cuda") for n in (cols, rows))
    s = torch.cuda.Stream()

    def run(side):
        now = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(now)
        h = cbk.ffn_gated(a, b, X, stream=side)
        y = cbk.linear(a, X)
        dx = cbk.ffn_gated_bwd(a, b, X, dH, stream=side)[0]
        if side is not None:
            now.wait_stream(side)
        return h, y, dx, h.float() + y.float()

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        outs = run(s)
    for i in range(4):
        X.copy_(acts(torch, T, cols, 120 + i))
        dH.copy_(acts(torch, T, rows, 130 + i, 0.1))
        g.replay()
        want = run(None)
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w), i
