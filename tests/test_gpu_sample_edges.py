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


def ends(torch, z, top_k, top_p=1.0):
    """The first and the last kept entry of a row by index, and their logprobs, as the header words them (the reference's
    running sum may seem to pass the whole one by what rounding leaves)."""
    order = sorted(range(len(z)), key=lambda i: (-z[i], i))[:top_k]
    p = [math.exp(z[i] - z[order[0]]) for i in order]
    n = len(p) if top_p >= 1 else next(n for n in range(1, len(p) + 1) if math.fsum(p[:n]) >= top_p * math.fsum(p))
    whole = math.log(math.fsum(p[:n]))
    return [(i, z[i] - z[order[0]] - whole) for i in (min(order[:n]), max(order[:n]))]


@pytest.mark.parametrize("T,V", [(3, 3000), (3, 9000), (3, 70000), (66, 70000)])
@pytest.mark.parametrize("low,spread", [(-200.0, 0.0), (-60.0, 2.5), (-30.0, 1.0)])
def test_a_uniform_number_at_and_past_its_ends(env, T, V, low, spread):
    """Twelve entries, and the rest far below them, of which top_k keeps a few: numbers up to 0 draw the first kept entry, those
    from 1 on the last, also where they weigh nothing beside the others, and never one that is left out."""
    torch, cbk = env
    g = torch.Generator().manual_seed(56)
    z = low + spread * torch.randn(3, V, generator=g)
    z[:, 1100:1112] = torch.randn(3, 12, generator=g)
    z[1, ::2] -= 100.0
    many = lambda v: v.repeat((T + 2) // 3, 1)[:T]
    for kw in ({"top_k": 20}, {"top_k": 1000}, {"top_k": 2000}, {"top_k": 13, "top_p": 0.9}, {"top_k": 2900}):
        want = [ends(torch, row, **kw) for row in z.tolist()]
        for v in (0.0, -1.0, math.nan, 1.0, 3.0):
            token, logprob = cbk.sample(many(z).cuda(), torch.full((T,), v, device="cuda"), **kw)
            for t in range(T):
                i, log = want[t % 3][1 if v >= 1 else 0]
                assert int(token[t]) == i, (kw, v, t, int(token[t]), i)
                assert abs(float(logprob[t]) - log) <= 2.0 ** -24 * abs(log) + 1e-11
        check(torch, cbk, z, torch.tensor([0.5, 0.01, 1.0 - 2.0 ** -24]), str(kw), **kw)


@pytest.mark.parametrize("T,V", [(3, 40000), (3, 70000), (66, 70000)])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -3.4028234663852886e38])
def test_masked_rows_at_the_ends_of_uniform(env, T, V, mask):
    """Fewer entries are allowed than top_k takes: the first or the last of them is drawn, for a few passes over the row (what is
    masked weighs nothing, so that no cut among it has to be found)."""
    torch, cbk = env
    g = torch.Generator().manual_seed(57)
    z = torch.full((T, V), mask)
    allowed = torch.randperm(V, generator=g)[:30]
    z[:, allowed] = 2.5 * torch.randn(T, 30, generator=g)
    z, plain = z.cuda(), 2.5 * torch.randn(T, V, generator=g).cuda()
    inside, ends = (torch.full((T,), v, device="cuda") for v in (0.5, 0.0))

    def us(x, u):
        times = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            cbk.sample(x, u, top_k=50)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return min(times)

    for v, want in ((0.0, allowed.min()), (-2.0, allowed.min()), (1.0, allowed.max()), (9.0, allowed.max())):
        token, logprob = cbk.sample(z, torch.full((T,), v, device="cuda"), top_k=50)
        assert bool((token == int(want)).all()) and bool(logprob.isfinite().all()), v
    ordinary, at_end = us(plain, inside), us(z, ends)
    assert at_end < 10 * ordinary, (ordinary, at_end)
