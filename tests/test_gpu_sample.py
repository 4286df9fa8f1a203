"""GPU tests of cbk_sample.h against a plain reference in 64 bits (moe_reference.sample): the token has to be the same."""
import math

import pytest

import moe_reference as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


def check(torch, cbk, z, u, what="", **settings):
    """`settings`: numbers, or lists with one for each row."""
    T = z.shape[0]
    given = {}
    for name, v in settings.items():
        given[name] = torch.tensor(v, dtype=torch.int32 if name == "top_k" else torch.float32).cuda() if isinstance(v, list) else v
    token, logprob = cbk.sample(z.cuda(), u.cuda(), **given)
    token, logprob = token.cpu().tolist(), logprob.cpu().tolist()
    for t in range(T):
        row = {name: float(torch.tensor(v[t] if isinstance(v, list) else v, dtype=torch.float32)) for name, v in settings.items()}
        row.setdefault("temperature", 1.0)
        want, log = moe.sample(z[t].tolist(), float(u[t]), **row)
        assert token[t] == want, (what, t, row, token[t], want)
        if math.isnan(log):
            assert math.isnan(logprob[t])
        else:  # formed in 64 bits and rounded once
            assert abs(logprob[t] - log) <= 2.0 ** -24 * abs(log) + 1e-11, (what, t, logprob[t], log)


def draws(torch, T, V, dtype, seed, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    z = spread * torch.randn(T, V, generator=g)
    z[torch.rand(T, V, generator=g) < 0.02] = -math.inf
    z[:, V // 2] = 0.5
    return z.to(dtype), torch.rand(T, generator=g)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [1, 2, 5, 64, 255, 1000, 4099, 33000])
def test_sample(env, V, dtype):
    torch, cbk = env
    T = 12
    z, u = draws(torch, T, V, getattr(torch, dtype), 1)
    check(torch, cbk, z, u, "temperature", temperature=0.8)
    check(torch, cbk, z, u, "greedy", temperature=0.0)
    for k in (1, 7, 50, 2500):
        check(torch, cbk, z, u, "top_k", top_k=k)
    for p in (0.0, 0.3, 0.9, 0.999):
        check(torch, cbk, z, u, "top_p", temperature=1.3, top_p=p)
    for m in (1e-6, 0.05, 1.0, 2.0):
        check(torch, cbk, z, u, "min_p", min_p=m)
    check(torch, cbk, z, u, "all", temperature=[0.0, 0.5, 1.0, 2.0, 1e-3, 50.0] * 2, top_k=[0, 3, 40, -1] * 3, top_p=[0.5, 0.95, 1.0] * 4,
          min_p=[0.0, 0.01, 0.2, 0.0, 0.001, 0.0] * 2)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sample_ties(env, dtype):
    """Many equal logits: a cut in the middle of them goes by index, also where they are too many to sort."""
    torch, cbk = env
    g = torch.Generator().manual_seed(2)
    z = torch.randint(-3, 4, (10, 9000), generator=g).float()
    z[0] = 1.0
    z[1] = 0.0
    z[1, ::3] = -0.0
    u = torch.rand(10, generator=g)
    z = z.to(getattr(torch, dtype))
    for kw in ({"top_k": 100}, {"top_k": 2000}, {"top_k": 8999}, {"top_p": 0.1}, {"top_p": 0.7, "top_k": 3000}, {"top_p": 0.5, "min_p": 0.3}):
        check(torch, cbk, z, u, str(kw), **kw)


def test_sample_extremes(env):
    torch, cbk = env
    low, inf = torch.finfo(torch.float32).min, math.inf
    z = torch.randn(14, 300, generator=torch.Generator().manual_seed(3))
    z[0] = -inf
    z[1] = -inf
    z[1, 299] = 3.0
    z[2] = low
    z[3, 10:] = low
    z[4, 7] = math.nan
    z[5, 3] = inf
    z[6, 5:9] = inf
    z[7] = -inf
    z[7, 0] = low
    z[8] *= 1e4
    z[9] *= 1e-30
    z[10] = torch.linspace(-80, 0, 300)
    z[11, 100] = 1e30
    z[12, 50:] = -inf
    z[13] = -1e38
    u = torch.rand(14, generator=torch.Generator().manual_seed(4))
    for kw in ({}, {"temperature": 0.0}, {"top_k": 5}, {"top_p": 0.5}, {"min_p": 0.1}, {"temperature": 1e-20, "top_p": 0.9},
               {"temperature": inf, "top_p": 0.4}, {"temperature": math.nan}, {"top_k": 200, "top_p": 0.99, "min_p": 1e-8}):
        check(torch, cbk, z, u, str(kw), **kw)


def test_sample_uniform_at_its_ends(env):
    torch, cbk = env
    z, _ = draws(torch, 8, 3000, torch.float32, 5)
    for v in (0.0, 1.0 - 2.0 ** -24, 1.0, 7.0, -1.0, math.nan):
        u = torch.full((8,), v)
        check(torch, cbk, z, u, v)
        check(torch, cbk, z, u, v, top_k=20, top_p=0.8)


def test_sample_rows_anywhere(env):
    """Rows that start on any element, with a stride; what surrounds them is not read."""
    torch, cbk = env
    for dtype in (torch.float32, torch.bfloat16):
        z, u = draws(torch, 9, 701, dtype, 6)
        for at in range(5):
            big = torch.full((9, 713), math.nan, dtype=dtype)
            big[:, at: at + 701] = z
            d = big.cuda()
            got = cbk.sample(d[:, at: at + 701], u.cuda(), top_k=50, top_p=0.9)
            want = cbk.sample(z.cuda(), u.cuda(), top_k=50, top_p=0.9)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_sample_the_largest_vocabulary(env):
    torch, cbk = env
    V = 1 << 20
    z, u = draws(torch, 3, V, torch.float32, 7)
    token, logprob = cbk.sample(z.cuda(), u.cuda())
    p = torch.softmax(z.double(), 1)
    c = p.cumsum(1)
    want = (c <= u.double()[:, None] * c[:, -1:]).sum(1)
    assert torch.equal(token.cpu(), want)
    assert bool(((logprob.cpu().double() - p.gather(1, want[:, None]).log()[:, 0]).abs() < 2e-6).all())
    got, _ = cbk.sample(z.cuda(), u.cuda(), top_k=3)
    assert bool((z.gather(1, got.cpu()[:, None]) >= z.topk(3)[0][:, -1:]).all())


def test_sample_draws_as_often_as_its_probabilities(env):
    torch, cbk = env
    z = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5])
    n = 20000
    u = (torch.arange(n) + 0.5) / n  # evenly over [0, 1)
    token, _ = cbk.sample(z.expand(n, 5).contiguous().cuda(), u.cuda(), temperature=0.7)
    share = torch.bincount(token.cpu(), minlength=5) / n
    assert bool(((share - torch.softmax(z / 0.7, 0)).abs() <= 1.5 / n).all())  # each interval's ends


@pytest.mark.parametrize("V", [60000, 70000])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sample_flat_rows(env, dtype, V):
    """Large vocabularies of nearly equal logits, whose cut lies among tens of thousands of entries of one bin."""
    torch, cbk = env
    g = torch.Generator().manual_seed(8)
    z = 1e-3 * torch.randn(3, V, generator=g)
    z[1] = torch.randint(0, 3, (V,), generator=g) * 2.0 ** -9
    z[2, 30000:] += 4.0
    z, u = z.to(getattr(torch, dtype)), torch.rand(3, generator=g)
    for kw in ({"top_p": 0.5}, {"top_k": 30000}, {"top_k": 29999, "top_p": 0.7}, {"top_p": 0.999, "min_p": 0.9}, {"temperature": 1e-3, "top_p": 0.3}):
        check(torch, cbk, z, u, str(kw), **kw)


def test_sample_many_rows(env):
    torch, cbk = env
    z, u = draws(torch, 700, 300, torch.bfloat16, 9)
    check(torch, cbk, z, u, temperature=0.9, top_k=20, top_p=0.8)
    T = (1 << 22) + 7
    z = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    z[-1] = -math.inf
    token, logprob = cbk.sample(z, torch.zeros(T, device="cuda"), top_k=torch.ones(T, dtype=torch.int32, device="cuda"))
    assert bool((token[:-1] == 0).all()) and bool((logprob[:-1] == 0).all()) and int(token[-1]) == -1 and bool(logprob[-1].isnan())


def test_sample_in_graphs_on_streams_and_without_logprob(env):
    """Replays with new inputs against eager calls; calls on another stream beside pending work; the C call's NULL."""
    import ctypes
    torch, cbk = env
    T, V = 40, 5000
    Z, U = torch.empty(T, V, device="cuda"), torch.empty(T, device="cuda")
    temperatures = torch.linspace(0, 2, T).cuda()

    def run(stream=None):
        return [*cbk.sample(Z, U, stream=stream), *cbk.sample(Z, U, temperature=temperatures, top_k=90, top_p=0.9, min_p=0.01, stream=stream)]

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    big, s = torch.ones(1 << 28, device="cuda"), torch.cuda.Stream()
    for i in range(4):
        z, u = draws(torch, T, V, torch.float32, 10 + i)
        Z.copy_(z)
        U.copy_(u)
        g.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
        for _ in range(10):
            big.mul_(1.0)
        side, here = run(s), run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(side, want, here)), i
    token = torch.full((T + 2,), 7, dtype=torch.int64, device="cuda")
    need = cbk.sample_workspace_bytes(T, V)
    whole = torch.empty(512 + need + 512, dtype=torch.uint8, device="cuda")
    assert cbk.sample_workspace_bytes(T, V, top_k=50) == 0
    for p, ws, n, expect in ((cbk._Sampling(1.0, 1.0, 0.0, 0), whole[512:].data_ptr(), need, want[0]),
                             (cbk._Sampling(1.0, 1.0, 0.0, 50), None, 0, cbk.sample(Z, U, top_k=50)[0])):
        whole.fill_(0x7F)
        token.fill_(7)
        assert cbk.load_library().cbk_sample(ctypes.byref(p), Z.data_ptr(), 0, V, V, T, U.data_ptr(), token[1:].data_ptr(), None, ws, n,
                                             torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(token[1:-1], expect) and int(token[0]) == 7 and int(token[-1]) == 7
        assert bool((whole[:512] == 0x7F).all()) and bool((whole[512 + need:] == 0x7F).all())


@pytest.mark.parametrize("spread", [0.0, 0.6])
def test_sample_a_cut_far_below_the_largest(env, spread):
    """One large logit and a million some e^-30 of it, whose sum 1 - top_p cuts into: what is kept of them shows in the
    logarithm of the large one's probability."""
    torch, cbk = env
    V = 1 << 20
    g = torch.Generator().manual_seed(11)
    z = -30.0 + spread * torch.rand(2, V, generator=g)
    z[:, V - 1] = 0.0
    u = torch.tensor([0.5, 2.0 ** -26])
    check(torch, cbk, z, u, top_p=1 - 2.0 ** -24)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [1, 3, 1021, 1024, 1025, 5000, 50257])
def test_sample_without_filters_by_numbers_and_by_vectors(env, V, dtype):
    """Numbers that filter nothing, and vectors of such numbers, are done by different kernels: rows from any element, every
    kind of temperature."""
    torch, cbk = env
    T, inf = 11, math.inf
    z, u = draws(torch, T, V, getattr(torch, dtype), 21)
    z[1] = -inf
    z[2, V // 2] = math.nan
    z[3, V - 1] = inf
    z[4, : V // 2 + 1] = inf
    z[5] = 0.0
    z[6, -1] = 60.0
    u[7], u[8], u[9] = 0.0, 1.0, math.nan
    for at in (0, 1, 3):
        big = torch.full((T, V + 7), math.nan, dtype=z.dtype)
        big[:, at: at + V] = z
        view = big.cuda()[:, at: at + V]
        for heat in (1.0, 0.0, -1.0, 0.3, inf, math.nan, 1e-30, torch.tensor([1.0, 0.5, 2.0, 1.0, 0.0, 0.7, 1.0, inf, 0.9, 1.1, math.nan]).cuda()):
            token, logprob = cbk.sample(view, u.cuda(), temperature=heat)
            same, close = cbk.sample(view, u.cuda(), temperature=heat, top_k=torch.zeros(T, dtype=torch.int32, device="cuda"),
                                     top_p=torch.full((T,), math.nan, device="cuda"), min_p=torch.full((T,), math.nan, device="cuda"))
            assert torch.equal(token, same), heat
            assert torch.equal(logprob.isnan(), close.isnan())
            ok = ~logprob.isnan()  # each formed in 64 bits and rounded once
            assert bool(((logprob - close).abs()[ok] <= 2.0 ** -23 * logprob.abs()[ok] + 1e-11).all()), heat
    for heat in (1.0, 0.0, inf):
        check(torch, cbk, z, u, heat, temperature=heat)


def test_sample_long_rows_with_filters(env):
    """Rows whose filters' work is divided: replayed with new inputs, on another stream beside pending work, with a workspace
    whose contents and surroundings do not matter; against the reference."""
    torch, cbk = env
    T, V = 61, 70001
    Z, U = torch.empty(T, V, dtype=torch.bfloat16, device="cuda"), torch.empty(T, device="cuda")
    g = torch.Generator().manual_seed(31)
    pick = lambda *values: torch.tensor(values)[torch.randint(0, len(values), (T,), generator=g)]
    kw = {"temperature": pick(0.0, 0.7, 1.0, 1.5), "top_k": pick(0, 1, 40, 1500, 4000, 9000).int(), "top_p": pick(1.0, 0.3, 0.95), "min_p": pick(0.0, 0.0, 0.05)}
    device = {n: v.cuda() for n, v in kw.items()}
    need = cbk.sample_workspace_bytes(T, V, **{n: device[n] for n in ("top_k", "top_p", "min_p")})
    assert need > 0
    whole = torch.empty(512 + need + 512, dtype=torch.uint8, device="cuda")
    graph, big, s = torch.cuda.CUDAGraph(), torch.ones(1 << 28, device="cuda"), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        outs = cbk.sample(Z, U, **device)
    for i in range(3):
        z, u = draws(torch, T, V, torch.bfloat16, 32 + i)
        Z.copy_(z)
        U.copy_(u)
        graph.replay()
        whole.fill_((0xFF, 0x00, 0x7F)[i])
        want = cbk.sample(Z, U, workspace=whole[512: 512 + need], **device)
        assert bool((whole[:512] == whole[0]).all()) and bool((whole[512 + need:] == whole[0]).all())
        for _ in range(10):
            big.mul_(1.0)
        side = cbk.sample(Z, U, stream=s, **device)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(outs, want, side)), i
    with pytest.raises(cbk.CbkError):
        cbk.sample(Z, U, workspace=whole[512: 512 + need - 1], **device)
    check(torch, cbk, z[:40], u[:40], **{n: v[:40].tolist() for n, v in kw.items()})
    # one workgroup a row, where there are more of them
    twice = [torch.cat([v, v]).cuda() for v in (z, u)]
    assert cbk.sample_workspace_bytes(2 * T, V, top_k=device["top_k"]) == 0
    token, logprob = cbk.sample(*twice, **{n: torch.cat([v, v]) for n, v in device.items()})
    assert torch.equal(token[:T], want[0]) and torch.equal(token[T:], want[0])
    a, b = logprob[:T], want[1]  # each formed in 64 bits and rounded once
    assert bool(((a - b).abs() <= 2.0 ** -23 * b.abs() + 1e-11).all())


def test_sample_long_rows_of_extremes(env):
    torch, cbk = env
    low, inf, V = torch.finfo(torch.float32).min, math.inf, 66001
    z = 2.5 * torch.randn(12, V, generator=torch.Generator().manual_seed(41))
    z[0] = -inf
    z[1] = -inf
    z[1, V - 1] = 3.0
    z[2] = low
    z[3, 10:] = low
    z[4, 7] = math.nan
    z[5, 3] = inf
    z[6, 5:66000:2] = inf
    z[7] *= 1e4
    z[8] *= 1e-30
    z[9, 65536:] = 90.0
    z[10, 50:] = -inf
    u = torch.rand(12, generator=torch.Generator().manual_seed(42))
    u[11] = 1.0
    for kw in ({"temperature": 0.0, "top_k": 3}, {"top_k": 5}, {"top_p": 0.5}, {"min_p": 0.1}, {"temperature": 1e-20, "top_p": 0.9},
               {"temperature": inf, "top_p": 0.4}, {"temperature": math.nan, "top_p": 0.4}, {"top_k": 2000, "top_p": 0.99, "min_p": 1e-8},
               {"top_p": 0.0}, {"top_k": 65999, "top_p": 0.6}, {"min_p": 0.3, "top_p": 0.6}, {"top_k": 1500, "min_p": 0.7}, {"min_p": 5.0}):
        check(torch, cbk, z, u, str(kw), **kw)
