"""GPU tests of the operators in include/cbk_nn.h at sizes where their way of computing changes: pieces of
the largest size that is decoded in the stream's order, several pieces, and the token tiles' limits."""
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


@pytest.mark.parametrize("rows,cols", [(32768, 4096), (40000, 4096), (300, 1 << 19)])
def test_a_piece_of_the_most_weights(env, rows, cols):
    """A piece of 2^27 weights, two pieces, and a piece of the fewest rows, with more tokens than are decoded on
    the way: some of the outputs, the last among them, against the reference."""
    torch, cbk = env
    T = 400
    g = torch.Generator(device="cuda").manual_seed(121)
    w = (torch.randn(rows, cols, generator=g, device="cuda") * 0.02).bfloat16()
    t = cbk.encode_gpu(w)
    at = torch.cat([torch.arange(0, rows, max(1, rows // 97)), torch.arange(rows - 40, rows)])
    part = w[at.cuda()].cpu()
    del w
    x, dy = acts(torch, T, cols, 122), torch.zeros(T, rows, dtype=torch.bfloat16)
    dy[:, at] = acts(torch, T, at.numel(), 123)
    y = cbk.linear(t, x.cuda()).cpu()
    ref.assert_within(y[:, at], *ref.linear(x, part), "linear")
    at, first = at.unique(return_inverse=True)
    rows_of = torch.empty(at.numel(), dtype=torch.long).scatter_(0, first, torch.arange(first.numel()))
    dx = cbk.linear_dx(t, dy.cuda())
    ref.assert_within(dx, *ref.linear_dx(dy[:, at], part[rows_of]), "linear_dx")
