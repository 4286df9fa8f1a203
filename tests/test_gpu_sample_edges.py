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


@pytest.mark.parametrize("V", [300, 5000, 66001])
@pytest.mark.parametrize("temperature", [1e-29, 1e-30, 3e-38, 7e-45])
def test_the_least_temperatures(env, temperature, V):
    """Logits that lie within some hundred temperatures of each other, down to where both are subnormal numbers."""
    torch, cbk = env
    g = torch.Generator().manual_seed(52)
    z = (2.5 * temperature * torch.randn(6, V, generator=g, dtype=torch.float64)).float()
    z[1] = 0.0
    z[2, ::2] = -1.0  # far away, like all that differ by more than their roundings
    z[3, 5:] = -math.inf
    u = torch.rand(6, generator=g)
    for kw in ({"top_p": 0.9}, {"top_p": 0.3}, {"top_k": 20}, {"top_k": 20, "top_p": 0.8}, {"min_p": 0.1}, {"min_p": 0.02, "top_p": 0.95}, {}):
        check(torch, cbk, z, u, str(kw), temperature=temperature, **kw)
    check(torch, cbk, z, u, "rows", temperature=[temperature, 1.0] * 3, top_p=[0.9, 0.5, 0.2] * 2)


def low_start(torch, T, V, mask, seed):
    """Rows whose first 4096 entries are masked by a finite number; of the others some are allowed."""
    g = torch.Generator().manual_seed(seed)
    z = 2.5 * torch.randn(T, V, generator=g)
    z[:, :4096] = mask
    z[1::2, 4096:-20] = mask  # 20 allowed entries
    return z, torch.rand(T, generator=g)


@pytest.mark.parametrize("mask", [-1e4, -1e9, -3.4028234663852886e38])
@pytest.mark.parametrize("T,V", [(4, 40000), (66, 70000)])
def test_masked_first_entries(env, T, V, mask):
    torch, cbk = env
    z, u = low_start(torch, 4, V, mask, 53)
    for kw in ({"top_k": 50}, {"top_k": 3000}, {"top_k": 50, "top_p": 0.9}, {"top_k": 3000, "top_p": 0.9}, {"top_k": 50, "min_p": 0.05}, {"top_p": 0.9}):
        check(torch, cbk, z.repeat((T + 3) // 4, 1)[:T] if kw == {"top_k": 50} else z, (u.repeat((T + 3) // 4))[:T] if kw == {"top_k": 50} else u, str(kw), **kw)


@pytest.mark.parametrize("kw", [{"top_k": 50}, {"top_k": 3000}, {"top_k": 50, "top_p": 0.9}])
def test_masked_first_entries_take_a_pass_more(env, kw):
    """A reference that is too low costs another pass over the row (in which much is added to one bin), not one for each of a
    key's 64 bits: less than 20 passes, where a row with nothing masked takes two."""
    torch, cbk = env
    T, V = 66, 70000
    z, u = low_start(torch, T, V, -1e9, 54)
    plain, _ = draws(torch, T, V, torch.float32, 55)
    z, plain, u = z.cuda(), plain.cuda(), u.cuda()

    def us(x):
        for _ in range(3):
            cbk.sample(x, u, **kw)
        times = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            cbk.sample(x, u, **kw)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return min(times)

    ordinary, masked = us(plain), us(z)
    assert masked < 10 * ordinary, (ordinary, masked)
