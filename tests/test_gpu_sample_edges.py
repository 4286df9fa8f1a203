"""GPU tests of cbk_sample.h at the ends of its settings and for masked rows, against the reference in 64 bits
(moe_reference.sample)."""
import math

import pytest

from test_gpu_sample import check, draws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


@pytest.mark.parametrize("V", [300, 66001])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_an_infinite_temperature_keeps_what_is_as_likely(env, dtype, V):
    """Every finite entry is as likely as the largest, so min_p leaves all of them, at its own end too."""
    torch, cbk = env
    z, u = draws(torch, 6, V, getattr(torch, dtype), 51)
    z[1] = torch.finfo(z.dtype).min
    z[1, V // 3] = 5.0
    z[2, : V // 2] = math.inf  # these alone count
    for kw in ({"min_p": 1.0}, {"min_p": 0.5}, {"min_p": 7.0}, {"min_p": 1.0, "top_k": 40}, {"min_p": 1.0, "top_p": 0.3}, {"min_p": 1.0, "top_k": 2500}):
        check(torch, cbk, z, u, str(kw), temperature=math.inf, **kw)
