"""GPU tests of the routing's gradient for experts that a bias or a limit on groups chose: not the largest logits, and fewer
than k where the kept groups run out."""
import math

import pytest

import moe_reference as moe
import nn_reference as ref
from test_gpu_moe import ROUTES, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,E,k,score,biased,groups,kept,top,renormalise",
                         [r for r in ROUTES if r[4] or r[5] > 1] + [(12, 32, 8, "softmax", False, 8, 1, 1, True), (12, 32, 8, "softmax", True, 8, 1, 2, False),
                                                                    (12, 30, 9, "sigmoid", True, 5, 1, 1, True), (40, 64, 8, "softmax", True, 1, 1, 1, False)])
def test_route_bwd_of_the_chosen(env, T, E, k, score, biased, groups, kept, top, renormalise, dtype):
    torch, cbk = env
    z = logits(torch, T, E, getattr(torch, dtype), 61)
    g = torch.Generator().manual_seed(62)
    bias = torch.randn(E, generator=g) if biased else None  # more than most scores differ by
    e, w = cbk.route(z.cuda(), k, score=score, bias=bias.cuda() if biased else None, groups=groups, top_groups=kept, group_top=top,
                     renormalise=renormalise, scale=0.7)
    we, _ = moe.route(z, k, score, bias, groups, kept, top, renormalise, 0.7)
    assert torch.equal(e.cpu(), we)
    if k > E // groups * kept:
        assert bool((we[:, -1] == -1).all())
    dw = torch.randn(T, k, generator=g)
    dw[we < 0] = math.nan  # of unused slots nothing is read
    dz = cbk.route_bwd(z.cuda(), e, dw.cuda(), score=score, renormalise=renormalise, scale=0.7)
    want, bound = moe.route_bwd(z, we, dw, score, renormalise, 0.7)
    ref.assert_within(dz, want, ref.rounded(want, bound) if dtype == "bfloat16" else bound, "dlogits")
