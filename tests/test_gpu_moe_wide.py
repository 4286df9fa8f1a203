"""GPU tests of blocks of experts (include/cbk_moe.h) with a million hidden columns and hundreds of experts in use, whose
products have more tiles than one launch may have."""
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


@pytest.mark.parametrize("patterns,count,T", [(2, 128, 128), (2, 600, 700), (9000, 600, 500)])
def test_a_million_hidden_columns(env, patterns, count, T):
    """Each token has an expert of its own, as far as they go; experts share three sets of tensors, and tokens eight rows of X,
    so that 24 rows of the reference are all there are."""
    torch, cbk = env
    rows, cols, out, sets, different = 1 << 20, 8, 8, 3, 8
    w = [[weights(torch, *shape, patterns, 100 * kind + i, 0.2) for i in range(sets)] for kind, shape in
         enumerate([(rows, cols), (rows, cols), (out, rows)])]
    ex = cbk.Experts(*([ts[e % sets] for e in range(count)] for ts in ([compress(cbk, t) for t in ts] for ts in w)))
    g = torch.Generator().manual_seed(32)
    x, by = acts(torch, different, cols, 31), torch.rand(different, 1, generator=g)
    which = torch.randint(0, different, (T,), generator=g)
    chosen = torch.cat([torch.randperm(count, generator=g) for _ in range(2)])[:T, None].int()
    y = cbk.ffn_experts(ex, x[which].cuda(), chosen.cuda(), by[which].cuda())
    each = torch.arange(different).repeat(sets)
    want, bound = moe.experts("silu", *w, x[each], torch.arange(sets).repeat_interleave(different)[:, None].int(), by[each])
    row = (chosen[:, 0] % sets) * different + which
    ref.assert_within(y, want[row], bound[row], "Y")
