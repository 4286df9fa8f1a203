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


def of_width(torch, rows, cols, b, seed):
    """BF16 weights whose index width is b (at most 15): as many finite patterns as it holds, less three,
    of falling exponents from 2^-4 on (2^-1 for 15 bits, whose patterns end at 32000); each occurs."""
    U = min(32000, max((1 << (b - 1)) + 1, (1 << b) - 3))
    top = 123 if b < 15 else 126
    i = torch.arange(U)
    patterns = (i & 1) << 15 | (top - (i >> 8)) << 7 | (i >> 1) & 127
    values = torch.where(patterns >= 1 << 15, patterns - (1 << 16), patterns).short().view(torch.bfloat16)
    g = torch.Generator().manual_seed(seed)
    w = values[torch.randint(0, U, (rows * cols,), generator=g)]
    w[torch.randperm(rows * cols, generator=g)[:U]] = values
    return w.reshape(rows, cols)


def every_operator(env, T, w, v, seed):
    """Each operator on W (and the pair W, V) against the reference."""
    torch, cbk = env
    rows, cols = w.shape
    a, b = compress(cbk, w), compress(cbk, v)
    x, dy = acts(torch, T, cols, seed), acts(torch, T, rows, seed + 1, 0.1)
    ref.assert_within(cbk.linear(a, x.cuda()), *ref.linear(x, w), "linear")
    ref.assert_within(cbk.linear_dx(a, dy.cuda()), *ref.linear_dx(dy, w), "linear_dx")
    ref.assert_within(cbk.ffn_gated(a, b, x.cuda()), *ref.ffn("silu", x, w, v), "ffn_gated")
    for name, got, want in zip(("dX", "dG", "dU"), cbk.ffn_gated_bwd(a, b, x.cuda(), dy.cuda()), ref.ffn_bwd("silu", x, w, v, dy)):
        ref.assert_within(got, *want, name)
    labels = torch.randint(0, rows, (T,), generator=torch.Generator().manual_seed(seed + 2))
    loss, lse = cbk.xent(a, x.cuda(), labels.cuda())
    (want, bound), (wl, bl) = ref.xent(x, w, labels, -100)
    ref.assert_within(loss, want, bound, "loss")
    ref.assert_within(lse, wl, bl, "lse")
    dx = cbk.xent_bwd(a, x.cuda(), labels.cuda(), lse, torch.ones(T).cuda())
    ref.assert_within(dx, *ref.xent_bwd(x, w, labels, torch.ones(T), -100), "dX of the head")
    return a, b


@pytest.mark.parametrize("T", [192, 193, 224, 255, 256, 257])
@pytest.mark.parametrize("rows,cols", [(700, 1088), (515, 1027), (260, 320)])
def test_14_bits_around_256_tokens(env, T, rows, cols):
    """The widest table beside the token tiles of 192, 256 and 320: rings of three and of two slices."""
    torch, _ = env
    a, b = every_operator(env, T, of_width(torch, rows, cols, 14, 124), of_width(torch, rows, cols, 14, 125), 126)
    assert a.b == 14 and b.b == 14


@pytest.mark.parametrize("b", range(1, 16))
@pytest.mark.parametrize("T", [1, 13, 45, 100, 192, 300, 400])
@pytest.mark.parametrize("rows,cols", [(515, 1088), (300, 1027)])
def test_every_width(env, T, rows, cols, b):
    """Whole units a row and ragged rows, at each token tile; the pair's second tensor is narrower by one bit
    at odd numbers of tokens."""
    torch, _ = env
    second = b - 1 if T % 2 and b > 1 else b
    a, c = every_operator(env, T, of_width(torch, rows, cols, b, 130), of_width(torch, rows, cols, second, 131), 132)
    assert a.b == b and c.b == second


@pytest.mark.parametrize("T,rows,cols,b,second", [(256, 40000, 64, 11, 11), (300, 30000, 1088, 12, 12), (128, 70000, 64, 11, 9)])
def test_a_block_decoded_on_the_way_in_pieces(env, T, rows, cols, b, second):
    """More rows than one piece's sums are kept for, one launch a pair and one a tensor."""
    torch, cbk = env
    wg, wu = of_width(torch, rows, cols, b, 141), of_width(torch, rows, cols, second, 142)
    x, dh = acts(torch, T, cols, 143), acts(torch, T, rows, 144, 0.1)
    g, u = compress(cbk, wg), compress(cbk, wu)
    assert (g.b, u.b) == (b, second)
    ref.assert_within(cbk.ffn_gated(g, u, x.cuda()), *ref.ffn("silu", x, wg, wu), "ffn_gated")
    for name, got, want in zip(("dX", "dG", "dU"), cbk.ffn_gated_bwd(g, u, x.cuda(), dh.cuda()), ref.ffn_bwd("silu", x, wg, wu, dh)):
        ref.assert_within(got, *want, name)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
@pytest.mark.parametrize("T", [300, 400, 600])
@pytest.mark.parametrize("b", [8, 11, 13, 14])
def test_activations_with_many_tokens(env, T, b, act):
    torch, cbk = env
    rows, cols = 515, 1088
    wg, wu = of_width(torch, rows, cols, b, 145), of_width(torch, rows, cols, b, 146)
    x, dh = acts(torch, T, cols, 147), acts(torch, T, rows, 148, 0.1)
    g, u = compress(cbk, wg), compress(cbk, wu)
    assert g.b == b == u.b
    ref.assert_within(cbk.ffn_gated(g, u, x.cuda(), act=act), *ref.ffn(act, x, wg, wu), "ffn_gated")
    got = cbk.ffn_gated_bwd(g, u, x.cuda(), dh.cuda(), act=act)
    for name, v, want in zip(("dX", "dG", "dU"), got, ref.ffn_bwd(act, x, wg, wu, dh)):
        ref.assert_within(v, *want, name)


@pytest.mark.parametrize("T,rows", [(200, 90000), (400, 40000)])
def test_labels_of_every_piece_and_of_none(env, T, rows):
    """A head in several pieces: first and last labels of the head, and the least and largest of all integers."""
    torch, cbk = env
    cols = 64
    w, x = of_width(torch, rows, cols, 10, 151), acts(torch, T, cols, 152)
    labels = torch.arange(T) * 1000003 % rows
    labels[0], labels[1], labels[2], labels[3], labels[4] = 0, rows - 1, rows // 2, -(1 << 63), (1 << 63) - 1
    none = torch.zeros(T, dtype=torch.bool)
    none[3:5] = True
    a = compress(cbk, w)
    loss, lse = (t.cpu() for t in cbk.xent(a, x.cuda(), labels.cuda()))
    dx = cbk.xent_bwd(a, x.cuda(), labels.cuda(), lse.cuda(), torch.ones(T).cuda()).cpu()
    assert bool(torch.isnan(loss[none]).all()) and bool(torch.isnan(dx[none]).all()) and bool(torch.isfinite(lse).all())
    x, labels = x[~none], labels[~none]
    ref.assert_within(loss[~none], *ref.xent(x, w, labels, -100)[0], "loss")
    ref.assert_within(dx[~none], *ref.xent_bwd(x, w, labels, torch.ones(len(labels)), -100), "dX")


@pytest.mark.parametrize("T", [1, 20, 300, 400])
def test_a_codebook_on_an_odd_element(env, T):
    """2-byte alignment is all that a codebook needs."""
    torch, cbk = env
    rows, cols = 300, 192
    w, v = of_width(torch, rows, cols, 11, 155), of_width(torch, rows, cols, 9, 156)

    def moved(t):
        cb = torch.zeros(t.U + 1, dtype=torch.int16, device="cuda")[1:]
        cb.copy_(t.codebook)
        return cbk.Compressed(t.rows, t.cols, t.U, t.b, cb, t.words)

    a, b = compress(cbk, w), moved(compress(cbk, v))
    x, dh = acts(torch, T, cols, 157), acts(torch, T, rows, 158, 0.1)
    ref.assert_within(cbk.linear(b, x.cuda()), *ref.linear(x, v), "linear")
    ref.assert_within(cbk.linear_dx(b, dh.cuda()), *ref.linear_dx(dh, v), "linear_dx")
    for g, u, wg, wu in ((a, b, w, v), (b, a, v, w)):
        ref.assert_within(cbk.ffn_gated(g, u, x.cuda()), *ref.ffn("silu", x, wg, wu), "ffn_gated")
        for name, got, want in zip(("dX", "dG", "dU"), cbk.ffn_gated_bwd(g, u, x.cuda(), dh.cuda()), ref.ffn_bwd("silu", x, wg, wu, dh)):
            ref.assert_within(got, *want, name)
