"""GPU tests of the operators in include/cbk_nn.h (products of any number of tokens, the gated
feed-forward block, the cross entropy of a compressed head, and their gradients) against plain
float64 references, within bounds that count the fp32 sums and BF16 roundings (nn_reference.py)."""
import pytest

import nn_reference as ref

pytestmark = pytest.mark.gpu

# (tokens, rows, cols, distinct patterns): sizes around the tiles', one of everything, ragged rows,
# every kind of width (0 bits, a few, the usual 12, all 16)
SHAPES = [
    (1, 1, 1, 1), (1, 64, 64, 200), (2, 17, 65, 3), (3, 300, 128, 4000), (16, 130, 192, 2), (17, 16, 64, 600),
    (33, 129, 100, 1000), (64, 256, 256, 5000), (65, 255, 321, 9000), (128, 128, 64, 1), (129, 100, 640, 300),
    (200, 515, 1000, 3000), (257, 384, 320, 40000), (31, 2000, 72, 30), (5, 700, 448, 20000),
]
# up to 384 tokens and widths 8 to 14 (all of them here), whole 64-field units a row and not: decoded on the way
FUSED = [
    (1, 128, 64, 250), (2, 1000, 1024, 500), (13, 515, 448, 1000), (16, 64, 4096, 2000), (17, 2113, 192, 4000),
    (63, 640, 1088, 8000), (64, 130, 64, 5000), (65, 384, 512, 16000), (128, 900, 320, 3000), (129, 1000, 576, 260),
    (200, 1291, 704, 16000), (256, 257, 2048, 7000),
    (257, 700, 129, 2000), (384, 260, 1001, 6000), (320, 384, 256, 10000), (12, 999, 333, 14000), (150, 129, 63, 300),
    (192, 65, 1025, 500), (7, 4097, 95, 1000),
]

# more tokens: pieces of the weights are decoded first; the first two share a tile's reduction among workgroups
MANY = [
    (500, 300, 20000, 3000), (385, 20000, 300, 2000), (600, 1000, 130, 40000), (1025, 515, 640, 900), (700, 129, 77, 5),
    (513, 33, 1088, 9000),
]


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


def weights(torch, rows, cols, U, seed, scale=0.05):
    """BF16 weights [rows][cols] (CPU) with at most U distinct patterns."""
    g = torch.Generator().manual_seed(seed)
    if U >= 30000:  # many exponents: more than 2^15 patterns
        w = torch.randn(rows, cols, generator=g, dtype=torch.float64) * 10.0 ** (torch.rand(rows, cols, generator=g) * 60 - 62)
        w = w.to(torch.bfloat16)
        w.view(-1)[:: 7] = (torch.randn(w.view(-1)[:: 7].numel(), generator=g) * scale).bfloat16()
        return w
    values = (torch.randn(U, generator=g) * scale).bfloat16()
    return values[torch.randint(0, U, (rows, cols), generator=g)]


def compress(cbk, w):
    return cbk.encode(w).to("cuda")


def acts(torch, T, n, seed, scale=1.0):
    return (torch.randn(T, n, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16()


@pytest.mark.parametrize("T,rows,cols,U", SHAPES + FUSED + MANY)
def test_linear(env, T, rows, cols, U):
    torch, cbk = env
    w, x = weights(torch, rows, cols, U, 1), acts(torch, T, cols, 2)
    y = cbk.linear(compress(cbk, w), x.cuda())
    ref.assert_within(y, *ref.linear(x, w), "linear")


@pytest.mark.parametrize("T,rows,cols,U", SHAPES + FUSED + MANY)
def test_linear_dx(env, T, rows, cols, U):
    torch, cbk = env
    w, dy = weights(torch, rows, cols, U, 3), acts(torch, T, rows, 4)
    dx = cbk.linear_dx(compress(cbk, w), dy.cuda())
    ref.assert_within(dx, *ref.linear_dx(dy, w), "linear_dx")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,rows,cols,U", SHAPES)
def test_ffn_gated(env, T, rows, cols, U, act):
    torch, cbk = env
    wg, wu, x = weights(torch, rows, cols, U, 5, 0.2), weights(torch, rows, cols, max(1, U // 3), 6, 0.2), acts(torch, T, cols, 7)
    h = cbk.ffn_gated(compress(cbk, wg), compress(cbk, wu), x.cuda(), act=act)
    ref.assert_within(h, *ref.ffn(act, x, wg, wu), "ffn_gated")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,rows,cols,U", SHAPES)
def test_ffn_gated_bwd(env, T, rows, cols, U, act):
    torch, cbk = env
    wg, wu, x = weights(torch, rows, cols, U, 8, 0.2), weights(torch, rows, cols, max(1, U // 3), 9, 0.2), acts(torch, T, cols, 10)
    dh = acts(torch, T, rows, 11, 0.1)
    got = cbk.ffn_gated_bwd(compress(cbk, wg), compress(cbk, wu), x.cuda(), dh.cuda(), act=act)
    for name, g, want in zip(("dX", "dG", "dU"), got, ref.ffn_bwd(act, x, wg, wu, dh)):
        ref.assert_within(g, *want, name)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,rows,cols,U", FUSED + MANY)
def test_ffn_pair_of_one_width(env, T, rows, cols, U, act):
    """Forward and gradient where gate and up have the same width (one launch decodes both)."""
    torch, cbk = env
    wg, x = weights(torch, rows, cols, U, 20, 0.2), acts(torch, T, cols, 22)
    wu = -wg.flip(0, 1)  # as many distinct patterns
    dh = acts(torch, T, rows, 23, 0.1)
    g, u = compress(cbk, wg), compress(cbk, wu)
    assert g.b == u.b
    ref.assert_within(cbk.ffn_gated(g, u, x.cuda(), act=act), *ref.ffn(act, x, wg, wu), "ffn_gated")
    got = cbk.ffn_gated_bwd(g, u, x.cuda(), dh.cuda(), act=act)
    for name, v, want in zip(("dX", "dG", "dU"), got, ref.ffn_bwd(act, x, wg, wu, dh)):
        ref.assert_within(v, *want, name)


@pytest.mark.parametrize("T,rows,cols,U", SHAPES + FUSED + MANY)
def test_xent_and_gradient(env, T, rows, cols, U):
    torch, cbk = env
    w, x = weights(torch, rows, cols, U, 12, 0.1), acts(torch, T, cols, 13)
    g = torch.Generator().manual_seed(14)
    labels = torch.randint(0, rows, (T,), generator=g)
    labels[T // 2:: 5] = -100
    labels[-1] = rows - 1
    dloss = torch.rand(T, generator=g) + 0.5
    d = compress(cbk, w)
    loss, lse = cbk.xent(d, x.cuda(), labels.cuda())
    (want, bound), (wlse, blse) = ref.xent(x, w, labels, -100)
    ref.assert_within(lse, wlse, blse, "lse")
    ref.assert_within(loss, want, bound, "loss")
    dx = cbk.xent_bwd(d, x.cuda(), labels.cuda(), lse, dloss.cuda())
    ref.assert_within(dx, *ref.xent_bwd(x, w, labels, dloss, -100), "dX")
    assert bool((dx[labels == -100] == 0).all())
