"""GPU tests of what the operators in include/cbk_nn.h do with faulty weights: a NaN or a corrupt index in
one row of one tensor shows in everything that is computed from that row, and in nothing else."""
import pytest

import nn_reference as ref
from test_gpu_nn import acts, compress, weights
from test_gpu_nn_edges import WAYS

pytestmark = pytest.mark.gpu

# and decoded first by the fast kernel, past the tokens that are decoded on the way
MORE = [(400, 300, 192, 3000)]


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


@pytest.mark.parametrize("which", ["gate", "up"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,rows,cols,U", WAYS + MORE)
def test_a_nan_in_one_tensor_of_the_block(env, T, rows, cols, U, act, which):
    """Only the gate's (or the up tensor's) row r holds a NaN: column r of H, dG and dU and all of dX are
    NaN, whatever the other projection gives; the other columns stay within their bounds."""
    torch, cbk = env
    wg, wu = weights(torch, rows, cols, U, 101, 0.2), weights(torch, rows, cols, U, 102, 0.2)
    x, dh = acts(torch, T, cols, 103), acts(torch, T, rows, 104, 0.1)
    r = rows // 3
    (wg if which == "gate" else wu)[r, cols // 2] = float("nan")
    g, u = compress(cbk, wg), compress(cbk, wu)
    h = cbk.ffn_gated(g, u, x.cuda(), act=act).cpu()
    dx, dg, du = (t.cpu() for t in cbk.ffn_gated_bwd(g, u, x.cuda(), dh.cuda(), act=act))
    assert bool(torch.isnan(h[:, r]).all()) and bool(torch.isnan(dg[:, r]).all())
    assert bool(torch.isnan(dx).all()) if which == "gate" else bool(torch.isnan(dx).any(1).all())
    # dU = dH act(g) does not depend on the up tensor
    assert bool(torch.isnan(du[:, r]).all()) == (which == "gate")
    keep = torch.arange(rows) != r
    wg[r], wu[r] = 0, 0
    ref.assert_within(h[:, keep], *(t[:, keep] for t in ref.ffn(act, x, wg, wu)), "H")
    _, *want = ref.ffn_bwd(act, x, wg, wu, dh)
    for name, got, (w, bound) in zip(("dG", "dU"), (dg, du), want):
        ref.assert_within(got[:, keep], w[:, keep], bound[:, keep], name)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T", [1, 20, 400])
def test_corrupt_gate_indices(env, T, act):
    """Gate indices at or past U read as 0x7FC0: the gradients of the rows that hold one are NaN, not zeros."""
    torch, cbk = env
    rows, cols, U = 96, 192, 300  # b = 9
    g = torch.Generator().manual_seed(105)
    words = torch.randint(-(1 << 31), 1 << 31, (cbk.words_for(rows * cols, 9),), generator=g).int()
    words = torch.where(torch.rand(words.shape, generator=g) < 0.995, 0, words).cuda()
    codebook = torch.arange(16000, 16000 + U).short().cuda()
    gate = cbk.Compressed(rows, cols, U, 9, codebook, words)
    bad = torch.isnan(cbk.decode_bf16(gate)).any(1).cpu()
    assert bool(bad.any()) and not bool(bad.all())
    up = compress(cbk, weights(torch, rows, cols, 300, 106, 0.2))
    x, dh = acts(torch, T, cols, 107), acts(torch, T, rows, 108, 0.1)
    h = cbk.ffn_gated(gate, up, x.cuda(), act=act).cpu()
    _, dg, du = (t.cpu() for t in cbk.ffn_gated_bwd(gate, up, x.cuda(), dh.cuda(), act=act))
    for t in (h, dg, du):
        assert torch.equal(torch.isnan(t), bad.expand(T, rows))
