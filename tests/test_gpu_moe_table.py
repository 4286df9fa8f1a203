"""GPU tests of the table that ``Experts`` makes: what it points to lives as long as it does."""
import weakref

import pytest

from test_gpu_moe import Block, routing
from test_gpu_nn import acts, compress, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


def test_the_arrays_stay_where_the_table_points(env):
    """A tensor whose arrays are replaced after the table was made."""
    torch, cbk = env
    b = Block(torch, cbk, 3, 130, 96, 70, [900, 4000])
    x = acts(torch, 20, 96, 41).cuda()
    chosen, w = (v.cuda() for v in routing(torch, 20, 3, 2, 42))
    before = cbk.ffn_experts(b.ex, x, chosen, w)
    arrays = []
    for t in (t for ts in b.ex.tensors for t in ts):
        arrays += [weakref.ref(t.words), weakref.ref(t.codebook)]
        other = compress(cbk, weights(torch, t.rows, t.cols, 50, 43))
        t.words, t.codebook, t.U, t.b = other.words, other.codebook, other.U, other.b
    assert all(a() is not None for a in arrays)
    torch.cuda.synchronize()
    filled = [torch.full((a().numel(),), 0x55, dtype=a().dtype, device="cuda") for a in arrays]  # what a freed one's memory would go to
    assert torch.equal(cbk.ffn_experts(b.ex, x, chosen, w), before) and len(filled) == len(arrays)
