"""GPU tests of the operators in include/cbk_moe.h (routing, blocks of experts over compressed tensors, and their
gradients) against plain float64 references, within bounds that count the fp32 sums and BF16 roundings
(moe_reference.py)."""
import math

import pytest

import moe_reference as moe
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


def logits(torch, T, E, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    z = 1.5 * torch.randn(T, E, generator=g)
    if T > 3:
        z[3] = -math.inf
    if T > 5:
        z[5, : E // 2] = -math.inf
    return z.to(dtype)


# (tokens, experts, k, score, bias, groups, kept, group_top, renormalise)
ROUTES = [
    (1, 1, 1, "softmax", False, 1, 1, 1, True), (1, 64, 8, "softmax", False, 1, 1, 1, True), (7, 5, 5, "sigmoid", False, 1, 1, 1, False),
    (33, 61, 5, "softmax", False, 1, 1, 1, False), (9, 65, 64, "softmax", False, 1, 1, 1, True), (130, 128, 8, "softmax", True, 1, 1, 1, True),
    (20, 256, 8, "sigmoid", True, 8, 4, 2, True), (20, 160, 6, "softmax", False, 8, 3, 1, True), (20, 160, 6, "softmax", False, 8, 3, 2, False),
    (10, 96, 4, "sigmoid", True, 96, 7, 2, True), (6, 1000, 3, "softmax", False, 2, 1, 2, True), (6, 1024, 64, "sigmoid", True, 4, 2, 1, False),
    (10, 24, 4, "sigmoid", False, 3, 2, 1, True), (8, 512, 10, "softmax", True, 64, 60, 2, True),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,E,k,score,biased,groups,kept,top,renormalise", ROUTES)
def test_route(env, T, E, k, score, biased, groups, kept, top, renormalise, dtype):
    torch, cbk = env
    z = logits(torch, T, E, getattr(torch, dtype), 1)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(2)) if biased else None
    e, w = cbk.route(z.cuda(), k, score=score, bias=bias.cuda() if biased else None, groups=groups, top_groups=kept, group_top=top,
                     renormalise=renormalise, scale=2.5)
    we, ww = moe.route(z, k, score, bias, groups, kept, top, renormalise, 2.5)
    assert torch.equal(e.cpu(), we)
    # weights are formed in 64 bits, to some 1e-13 of themselves, and rounded once
    assert bool(((w.double().cpu() - ww).abs() <= (U := 2.0 ** -24) * ww.abs() * 1.001 + 2.0 ** -149).all()), U


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,E,k,score,biased,groups,kept,top,renormalise", ROUTES)
def test_route_bwd(env, T, E, k, score, biased, groups, kept, top, renormalise, dtype):
    torch, cbk = env
    z = logits(torch, T, E, getattr(torch, dtype), 3)
    g = torch.Generator().manual_seed(4)
    e, _ = cbk.route(z.cuda(), k, score=score, renormalise=renormalise)
    dw = torch.randn(T, k, generator=g)
    dz = cbk.route_bwd(z.cuda(), e, dw.cuda(), score=score, renormalise=renormalise, scale=0.7)
    want, bound = moe.route_bwd(z, e, dw, score, renormalise, 0.7)
    assert dz.dtype == z.dtype
    ref.assert_within(dz, want, ref.rounded(want, bound) if dtype == "bfloat16" else bound, "dlogits")


def test_route_ties_go_to_the_lower_index(env):
    torch, cbk = env
    z = torch.randint(-2, 3, (50, 96), generator=torch.Generator().manual_seed(5)).float() * 0.5
    z[0] = 0.0
    z[1, ::2] = -0.0
    z[1, 1::2] = 0.0
    for kw in ({}, {"groups": 12, "top_groups": 5}, {"groups": 12, "top_groups": 5, "group_top": 2}, {"score": "sigmoid"},
               {"bias": torch.zeros(96)}, {"bias": torch.zeros(96), "groups": 8, "top_groups": 3, "score": "sigmoid"}):
        want, _ = moe.route(z, 6, **kw)
        got, _ = cbk.route(z.cuda(), 6, **{n: v.cuda() if n == "bias" else v for n, v in kw.items()})
        assert torch.equal(got.cpu(), want), kw


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_rows_that_are_masked_or_broken(env, score, biased):
    torch, cbk = env
    inf, low = math.inf, torch.finfo(torch.float32).min
    z = torch.randn(12, 10, generator=torch.Generator().manual_seed(6))
    z[0] = -inf
    z[1, 1:] = -inf
    z[2] = low
    z[3, 4:] = low
    z[4, 2] = math.nan
    z[5, 9] = inf
    z[6] = 200.0
    z[7] = -200.0 - torch.arange(10)
    z[8, :] = -inf
    z[8, 7] = low
    bias = None
    if biased:
        bias = torch.zeros(10)
        bias[3] = -inf
        bias[6] = inf
    for renormalise in (True, False):
        e, w = cbk.route(z.cuda(), 4, score=score, bias=bias.cuda() if biased else None, renormalise=renormalise)
        we, ww = moe.route(z, 4, score, bias, renormalise=renormalise)
        assert torch.equal(e.cpu(), we)
        assert torch.equal(w.cpu().isnan(), ww.isnan())
        ok = ~ww.isnan()
        assert bool(((w.double().cpu() - ww).abs()[ok] <= 2.0 ** -23 * ww[ok] + 2.0 ** -149).all())
        dz = cbk.route_bwd(z.cuda(), e, torch.ones(12, 4, device="cuda"), score=score, renormalise=renormalise).cpu()
        assert bool(dz[4].isnan().all()) and bool(dz[5].isnan().all())
        assert bool((dz[[0]] == 0).all()) and bool(dz[[1, 2, 3, 6, 7, 8]].isfinite().all())


def test_route_reads_and_writes_only_its_rows(env):
    torch, cbk = env
    big = torch.full((40, 100), math.nan)
    big[3:23, 5:66] = logits(torch, 20, 61, torch.float32, 7)
    for dtype in (torch.float32, torch.bfloat16):
        d = big.to(dtype).cuda()
        view = d[3:23, 5:66]
        e, w = cbk.route(view, 3)
        e2, w2 = cbk.route(view.contiguous(), 3)
        assert torch.equal(e, e2) and torch.equal(w, w2)
        out = torch.full((22, 90), 7.0, dtype=dtype, device="cuda")
        cbk.route_bwd(view, e, w, out=out[1:21, 3:64])
        inside = torch.zeros_like(out, dtype=torch.bool)
        inside[1:21, 3:64] = True
        assert bool((out[~inside] == 7).all())
        assert torch.equal(out[1:21, 3:64], cbk.route_bwd(view.contiguous(), e, w))


def test_route_bwd_the_same_expert_twice_and_none(env):
    torch, cbk = env
    z = torch.randn(6, 9, generator=torch.Generator().manual_seed(8))
    e = torch.tensor([[2, 2, 5], [-1, 3, 3], [9, 8, 1], [-1, -1, -1], [0, 0, 0], [-7, 100, 4]], dtype=torch.int32)
    dw = torch.randn(6, 3, generator=torch.Generator().manual_seed(9))
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            got = cbk.route_bwd(z.cuda(), e.cuda(), dw.cuda(), score=score, renormalise=renormalise)
            ref.assert_within(got, *moe.route_bwd(z, e, dw, score, renormalise), (score, renormalise))


@pytest.mark.parametrize("score,renormalise", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_bwd_against_differences(env, score, renormalise):
    torch, cbk = env
    z = torch.randn(5, 12, generator=torch.Generator().manual_seed(10))
    z[:, :3] += 4  # the three chosen stay chosen
    dw = torch.randn(5, 3, generator=torch.Generator().manual_seed(11))
    e, _ = cbk.route(z.cuda(), 3, score=score, renormalise=renormalise)
    dz = cbk.route_bwd(z.cuda(), e, dw.cuda(), score=score, renormalise=renormalise).double().cpu()
    step = 1e-4

    def value(v):
        we, ww = moe.route(v, 3, score, renormalise=renormalise)
        assert torch.equal(we, e.cpu())
        return (ww * dw.double()).sum()
    for i in range(5):
        for j in range(12):
            d = torch.zeros(5, 12, dtype=torch.float64)
            d[i, j] = step
            slope = float((value(z.double() + d) - value(z.double() - d)) / (2 * step))
            # third derivatives of the scores are below 1, the gradients' sum below 10: 10 step^2 / 6, and fp32 roundings
            assert abs(slope - float(dz[i, j])) < 1e-6 + 2e-6, (i, j)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_route_scores_far_below_one(env, score, dtype):
    """Logits whose sigmoids are nothing in fp32, and nothing in fp64: renormalised weights and their gradient are not."""
    torch, cbk = env
    g = torch.Generator().manual_seed(12)
    low = torch.tensor([-20.0, -29.5, -30.5, -60.0, -87.0, -95.0, -120.0, -300.0])[:, None]
    z = (low + 1.5 * torch.randn(8, 20, generator=g)).to(getattr(torch, dtype))
    dw = torch.randn(8, 4, generator=g)
    e, w = cbk.route(z.cuda(), 4, score=score)
    we, ww = moe.route(z, 4, score)
    assert torch.equal(e.cpu(), we) and bool(((w.cpu().double() - ww).abs() <= 2.0 ** -24 * 1.001 * ww).all())
    want, bound = moe.route_bwd(z, we, dw, score)
    dz = cbk.route_bwd(z.cuda(), e, dw.cuda(), score=score)
    ref.assert_within(dz, want, ref.rounded(want, bound) if dtype == "bfloat16" else bound, "dlogits")
    far = torch.tensor([[-800.0, -801.0, -900.0, -1e30], [-1e4, -1e4, -2e4, -1e4]])
    e, w = cbk.route(far.cuda(), 3, score=score)
    we, ww = moe.route(far, 3, score)
    # (e^-100 is a subnormal number, of which fp32 has the multiples of 2^-149: rounding is off by up to half of one)
    assert torch.equal(e.cpu(), we) and bool(((w.cpu().double() - ww).abs() <= 2.0 ** -24 * 1.001 * ww + 2.0 ** -150).all())
    assert bool(cbk.route_bwd(far.cuda(), e, torch.rand(2, 3).cuda(), score=score).isfinite().all())


def routing(torch, T, E, k, seed, unused=True):
    g = torch.Generator().manual_seed(seed)
    chosen = torch.rand(T, E, generator=g).topk(min(k, E), 1)[1]
    if k > E:
        chosen = torch.cat([chosen, chosen[:, : k - E]], 1)
    w = torch.rand(T, k, generator=g)
    if unused:
        chosen[torch.rand(T, k, generator=g) < 0.1] = -1
    return chosen.int(), w


class Block:
    def __init__(self, torch, cbk, E, rows, cols, out, patterns, seed=20):
        """`patterns`: distinct patterns of each tensor, in turn."""
        it = iter(range(10 ** 6))
        def make(r, c, s):
            return [weights(torch, r, c, patterns[next(it) % len(patterns)], s + i, 0.2 if r == rows else 0.1) for i in range(E)]
        self.wg, self.wu, self.wd = make(rows, cols, seed), make(rows, cols, seed + 100), make(out, rows, seed + 200)
        self.ex = cbk.Experts(*([compress(cbk, w) for w in ws] for ws in (self.wg, self.wu, self.wd)))


# (tokens, experts, k, rows, cols, out, patterns): one of everything, ragged sizes, every kind of width (alone and side by
# side), tiles that are full, begun and empty, more slots than a tile takes
BLOCKS = [
    (1, 1, 1, 1, 1, 1, [1]), (1, 4, 2, 64, 64, 64, [200]), (3, 5, 2, 100, 70, 33, [3, 300, 4000]), (17, 3, 2, 130, 192, 128, [1000, 9000]),
    (16, 8, 4, 128, 256, 256, [5000]), (40, 2, 1, 65, 129, 300, [2, 600]), (70, 3, 3, 300, 500, 200, [4000, 5000, 700]),
    (200, 2, 2, 96, 64, 160, [1, 16000]), (333, 3, 2, 191, 321, 100, [6000, 12000]), (600, 2, 1, 128, 128, 128, [300]),
    (900, 4, 2, 257, 65, 190, [3000, 5000]), (30, 40, 6, 64, 96, 64, [500, 50]), (25, 3, 2, 130, 80, 70, [20000, 300]),
    (20, 2, 2, 300, 300, 128, [40000, 20000]), (260, 1, 1, 640, 1024, 256, [8000]), (45, 7, 2, 683, 1001, 1001, [9000, 4000]),
    (5, 2, 4, 64, 128, 64, [100]),
    # long reductions: what one slice leaves in flight meets the next ones
    (6, 4, 2, 384, 4096, 700, [5000]), (2, 3, 2, 2048, 320, 2048, [9000, 5000]), (520, 2, 1, 192, 2048, 1500, [5000]),
]


@pytest.mark.parametrize("T,E,k,rows,cols,out,patterns", BLOCKS)
def test_experts(env, T, E, k, rows, cols, out, patterns):
    torch, cbk = env
    b = Block(torch, cbk, E, rows, cols, out, patterns)
    x = acts(torch, T, cols, 21)
    chosen, w = routing(torch, T, E, k, 22)
    y = cbk.ffn_experts(b.ex, x.cuda(), chosen.cuda(), w.cuda())
    ref.assert_within(y, *moe.experts("silu", b.wg, b.wu, b.wd, x, chosen, w), "Y")


@pytest.mark.parametrize("T,E,k,rows,cols,out,patterns", BLOCKS)
def test_experts_bwd(env, T, E, k, rows, cols, out, patterns):
    torch, cbk = env
    b = Block(torch, cbk, E, rows, cols, out, patterns)
    x, dy = acts(torch, T, cols, 23), acts(torch, T, out, 24, 0.1)
    chosen, w = routing(torch, T, E, k, 25)
    dx, dw = cbk.ffn_experts_bwd(b.ex, x.cuda(), chosen.cuda(), w.cuda(), dy.cuda())
    for name, got, want in zip(("dX", "dweights"), (dx, dw), moe.experts_bwd("silu", b.wg, b.wu, b.wd, x, chosen, w, dy)):
        ref.assert_within(got, *want, name)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
@pytest.mark.parametrize("T", [9, 300])
def test_experts_activations(env, T, act):
    torch, cbk = env
    b = Block(torch, cbk, 3, 200, 130, 90, [5000])
    x, dy = acts(torch, T, 130, 26), acts(torch, T, 90, 27, 0.1)
    chosen, w = routing(torch, T, 3, 2, 28)
    y = cbk.ffn_experts(b.ex, x.cuda(), chosen.cuda(), w.cuda(), act=act)
    ref.assert_within(y, *moe.experts(act, b.wg, b.wu, b.wd, x, chosen, w), "Y")
    got = cbk.ffn_experts_bwd(b.ex, x.cuda(), chosen.cuda(), w.cuda(), dy.cuda(), act=act)
    for name, g, want in zip(("dX", "dweights"), got, moe.experts_bwd(act, b.wg, b.wu, b.wd, x, chosen, w, dy)):
        ref.assert_within(g, *want, name)
