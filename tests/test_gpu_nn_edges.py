"""GPU tests of what the operators in include/cbk_nn.h promise at their edges: views and padding left
alone, infinities and NaN, empty sizes, several chunks and pieces, captured graphs, streams, corrupt
indices, tensors past 4 GB, and a block and a head run together with their gradients."""
import math

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


def bits(torch, x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.int32)


# tokens, rows, cols, patterns: one for each way a product is done (the GEMV, k_fused, ragged, decoded
# first and in whole tiles, decoded first by the generic kernel)
WAYS = [(1, 260, 256, 3000), (20, 260, 256, 3000), (20, 261, 131, 3000), (300, 260, 192, 3000), (30, 70, 128, 40000)]


def every(cbk, torch, T, rows, cols, U, X=None, dY=None, head=None):
    """name -> a call of each operator on a fixed problem, taking X [T][cols], dY [T][rows]."""
    w, v = weights(torch, rows, cols, U, 31, 0.1), weights(torch, rows, cols, U, 32, 0.1)
    a, b = compress(cbk, w), compress(cbk, v)
    g = torch.Generator().manual_seed(33)
    labels = torch.randint(0, rows, (T,), generator=g).cuda()
    dloss = torch.rand(T, generator=g).cuda()
    return {
        "linear": lambda X, dY: [cbk.linear(a, X)],
        "linear_dx": lambda X, dY: [cbk.linear_dx(a, dY)],
        "ffn_gated": lambda X, dY: [cbk.ffn_gated(a, b, X)],
        "ffn_gated_bwd": lambda X, dY: list(cbk.ffn_gated_bwd(a, b, X, dY)),
        "xent": lambda X, dY: list(cbk.xent(a, X, labels)),
        "xent_bwd": lambda X, dY: [cbk.xent_bwd(a, X, labels, cbk.xent(a, X, labels)[1], dloss)],
    }


@pytest.mark.parametrize("T,rows,cols,U", WAYS)
def test_views_give_the_same_bits(env, T, rows, cols, U):
    """Rows with padding, at 2-byte alignment, surrounded by NaN: the same results, bit for bit."""
    torch, cbk = env
    X, dY = acts(torch, T, cols, 34).cuda(), acts(torch, T, rows, 35).cuda()

    def view(x, pad, lead):
        big = torch.full((x.shape[0] + 2, x.shape[1] + pad + lead), float("nan"), dtype=x.dtype, device=x.device)
        big[1:-1, lead: lead + x.shape[1]] = x
        return big[1:-1, lead: lead + x.shape[1]]

    for name, call in every(cbk, torch, T, rows, cols, U).items():
        want = call(X, dY)
        for pad, lead in ((8, 0), (24, 8), (5, 3)):
            for got, w in zip(call(view(X, pad, lead), view(dY, pad, lead)), want):
                assert torch.equal(bits(torch, got), bits(torch, w)), (name, pad, lead)


@pytest.mark.parametrize("pad,lead", [(0, 0), (4, 4), (3, 1)])
@pytest.mark.parametrize("T,rows,cols,U", WAYS)
def test_outputs_leave_their_surroundings(env, T, rows, cols, U, pad, lead):
    torch, cbk = env
    w = weights(torch, rows, cols, U, 36, 0.1)
    a = compress(cbk, w)
    X, dY = acts(torch, T, cols, 37).cuda(), acts(torch, T, rows, 38).cuda()
    labels = torch.randint(0, rows, (T,), generator=torch.Generator().manual_seed(39)).cuda()
    loss, lse = cbk.xent(a, X, labels)
    ones = torch.ones(T, device="cuda")
    calls = [
        (rows, lambda out: cbk.linear(a, X, out=out)), (cols, lambda out: cbk.linear_dx(a, dY, out=out)),
        (rows, lambda out: cbk.ffn_gated(a, a, X, out=out)), (cols, lambda out: cbk.ffn_gated_bwd(a, a, X, dY, dX=out)[0]),
        (cols, lambda out: cbk.xent_bwd(a, X, labels, lse, ones, out=out)),
    ]
    for i, (width, call) in enumerate(calls):
        want = call(None)
        big = torch.full((T + 2, width + pad + lead), 7.0, dtype=torch.bfloat16, device="cuda")
        out = big[1:-1, lead: lead + width]
        call(out)
        assert torch.equal(bits(torch, out), bits(torch, want)), i
        out.fill_(7.0)
        assert bool((big == 7.0).all()), i


@pytest.mark.parametrize("T,rows,cols,U", WAYS)
def test_same_bits_again(env, T, rows, cols, U):
    torch, cbk = env
    X, dY = acts(torch, T, cols, 40).cuda(), acts(torch, T, rows, 41).cuda()
    for name, call in every(cbk, torch, T, rows, cols, U).items():
        want = [x.clone() for x in call(X, dY)]
        torch.empty(1 << 26, dtype=torch.uint8, device="cuda").fill_(0xFF)  # other contents in the next workspace
        for got, w in zip(call(X, dY), want):
            assert torch.equal(bits(torch, got), bits(torch, w)), name


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,rows,cols,U", WAYS)
def test_a_token_that_is_not_finite_stays_in_its_row(env, T, rows, cols, U, bad):
    torch, cbk = env
    X, dY = acts(torch, T, cols, 42).cuda(), acts(torch, T, rows, 43).cuda()
    at = T // 2
    X2, dY2 = X.clone(), dY.clone()
    X2[at, -1] = bad
    dY2[at, -1] = bad
    others = torch.arange(T, device="cuda") != at
    for name, call in every(cbk, torch, T, rows, cols, U).items():
        for got, want in zip(call(X2, dY2), call(X, dY)):
            assert torch.equal(bits(torch, got[others]), bits(torch, want[others])), name
            assert not bool(torch.isfinite(got[at]).all()), name


@pytest.mark.parametrize("T,rows,cols,U", WAYS)
def test_a_weight_that_is_not_finite(env, T, rows, cols, U):
    """An infinite last weight: its row's outputs forward, its column's gradients, nothing else."""
    torch, cbk = env
    w = weights(torch, rows, cols, min(U, 20000), 44, 0.1)
    w2 = w.clone()
    w2[-1, -1] = float("inf")
    # the patterns (and so the width) of both are the same number: the infinity replaces one that occurs once
    X, dY = acts(torch, T, cols, 45), acts(torch, T, rows, 46)
    X[:, -1], dY[:, -1] = 1.0, 1.0
    y, y2 = (cbk.linear(compress(cbk, t), X.cuda()).cpu() for t in (w, w2))
    ref.assert_within(y2[:, :-1], *(t[:, :-1] for t in ref.linear(X, w)), "linear")
    assert bool((y2[:, -1] == float("inf")).all()) and bool(torch.isfinite(y).all())
    d2 = cbk.linear_dx(compress(cbk, w2), dY.cuda()).cpu()
    ref.assert_within(d2[:, :-1], *(t[:, :-1] for t in ref.linear_dx(dY, w)), "linear_dx")
    assert bool((d2[:, -1] == float("inf")).all())


@pytest.mark.parametrize("T", [1, 20, 300])
def test_xent_of_infinite_and_lowest_logits(env, T):
    """cols == 1 and x == 1: the logits are the weights.  Masked rows of the vocabulary (-inf, and the type's
    lowest value) take no part; all masked gives -inf and a loss of NaN; +inf gives +inf."""
    torch, cbk = env
    V = 1000
    z = (torch.randn(V, generator=torch.Generator().manual_seed(47)) * 3).bfloat16()
    z[100:900] = -float("inf")
    z[900:950] = torch.finfo(torch.bfloat16).min
    X = torch.ones(T, 1, dtype=torch.bfloat16)
    labels = (torch.arange(T) * 7) % 100
    a = compress(cbk, z[:, None])
    loss, lse = (t.double().cpu() for t in cbk.xent(a, X.cuda(), labels.cuda()))
    want = torch.logsumexp(z.double(), 0)
    assert float((lse - want).abs().max()) <= 1100 * ref.U32 * 8
    assert float((loss - (want - z.double()[labels])).abs().max()) <= 1200 * ref.U32 * 8
    # labels in the masked part: an infinite loss, and the lowest value's
    loss, _ = cbk.xent(a, X.cuda(), torch.full((T,), 500).cuda())
    assert bool((loss == float("inf")).all())
    none = compress(cbk, torch.full((V, 1), -float("inf"), dtype=torch.bfloat16))
    loss, lse = cbk.xent(none, X.cuda(), labels.cuda())
    assert bool((lse == -float("inf")).all()) and bool(torch.isnan(loss).all())
    z[3] = float("inf")
    loss, lse = cbk.xent(compress(cbk, z[:, None]), X.cuda(), labels.cuda())
    assert bool((lse == float("inf")).all())


@pytest.mark.parametrize("T,rows,cols,U", WAYS)
def test_ignored_and_invalid_labels(env, T, rows, cols, U):
    torch, cbk = env
    w = weights(torch, rows, cols, U, 48, 0.1)
    a, X = compress(cbk, w), acts(torch, T, cols, 49)
    labels = torch.randint(0, rows, (T,), generator=torch.Generator().manual_seed(50))
    kinds = torch.arange(T) % 5
    labels[kinds == 1] = -7                       # ignored
    labels[kinds == 2] = rows                     # out of range
    labels[kinds == 3] = -(1 << 40)
    labels[kinds == 4] = (1 << 32) + 1            # in range if it were cut to 32 bits
    X[kinds == 1] = float("nan")
    loss, lse = cbk.xent(a, X.cuda(), labels.cuda(), ignore_index=-7)
    dloss = torch.ones(T).cuda()
    dloss[(kinds == 1).cuda()] = float("inf")
    dx = cbk.xent_bwd(a, X.cuda(), labels.cuda(), lse, dloss, ignore_index=-7).cpu()
    loss = loss.cpu()
    assert bool((loss[kinds == 1] == 0).all()) and bool((dx[kinds == 1] == 0).all())
    for k in (2, 3, 4):
        assert bool(torch.isnan(loss[kinds == k]).all()) and bool(torch.isnan(dx[kinds == k]).all())
    good = kinds == 0
    (want, bound), _ = ref.xent(X[good], w, labels[good], -7)
    ref.assert_within(loss[good], want, bound, "loss")
    ref.assert_within(dx[good], *ref.xent_bwd(X[good], w, labels[good], torch.ones(int(good.sum())), -7), "dX")


def test_empty_sizes(env):
    torch, cbk = env
    a = compress(cbk, weights(torch, 20, 64, 300, 51))
    empty = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert cbk.linear(a, empty(0, 64)).shape == (0, 20)
    assert cbk.linear_dx(a, empty(0, 20)).shape == (0, 64)
    assert cbk.ffn_gated(a, a, empty(0, 64)).shape == (0, 20)
    assert [t.shape[0] for t in cbk.ffn_gated_bwd(a, a, empty(0, 64), empty(0, 20))] == [0, 0, 0]
    loss, lse = cbk.xent(a, empty(0, 64), none)
    assert cbk.xent_bwd(a, empty(0, 64), none, lse, loss).shape == (0, 64)
    for T in (1, 40, 400):
        flat = cbk.encode(torch.zeros(20, 0, dtype=torch.bfloat16), 20, 0).to("cuda")  # no columns
        assert bool((cbk.linear(flat, empty(T, 0)) == 0).all()) and cbk.linear(flat, empty(T, 0)).shape == (T, 20)
        assert cbk.linear_dx(flat, empty(T, 20)).shape == (T, 0)
        assert bool((cbk.ffn_gated(flat, flat, empty(T, 0)) == 0).all())
        dx, dg, du = cbk.ffn_gated_bwd(flat, flat, empty(T, 0), torch.ones(T, 20, dtype=torch.bfloat16, device="cuda"))
        assert dx.shape == (T, 0) and bool((dg == 0).all()) and bool((du == 0).all())
        loss, lse = cbk.xent(flat, empty(T, 0), torch.zeros(T, dtype=torch.int64, device="cuda"))
        assert float((lse - math.log(20)).abs().max()) <= 64 * ref.U32 and float((loss - lse).abs().max()) == 0
        tall = cbk.encode(torch.zeros(0, 64, dtype=torch.bfloat16), 0, 64).to("cuda")  # no rows
        assert cbk.linear(tall, empty(T, 64)).shape == (T, 0)
        assert bool((cbk.linear_dx(tall, empty(T, 0)) == 0).all())
        assert bool((cbk.ffn_gated_bwd(tall, tall, empty(T, 64), empty(T, 0))[0] == 0).all())


@pytest.mark.parametrize("T,rows,cols,U", [(8200, 40, 70, 700), (300, 40000, 64, 700), (200, 90000, 64, 700)])
def test_chunks_of_tokens_and_pieces_of_rows(env, T, rows, cols, U):
    """More than 8192 tokens, more rows than a piece holds: decoded first (the first two), and on the way."""
    torch, cbk = env
    w, x, dy = weights(torch, rows, cols, U, 52, 0.1), acts(torch, T, cols, 53), acts(torch, T, rows, 54, 0.1)
    a = compress(cbk, w)
    ref.assert_within(cbk.linear(a, x.cuda()), *ref.linear(x, w), "linear")
    ref.assert_within(cbk.linear_dx(a, dy.cuda()), *ref.linear_dx(dy, w), "linear_dx")
    labels = torch.randint(0, rows, (T,), generator=torch.Generator().manual_seed(55))
    labels[::9] = -100
    loss, lse = cbk.xent(a, x.cuda(), labels.cuda())
    (want, bound), (wl, bl) = ref.xent(x, w, labels, -100)
    ref.assert_within(loss, want, bound, "loss")
    ref.assert_within(lse, wl, bl, "lse")
    dx = cbk.xent_bwd(a, x.cuda(), labels.cuda(), lse, torch.ones(T).cuda())
    ref.assert_within(dx, *ref.xent_bwd(x, w, labels, torch.ones(T), -100), "dX")
    if rows <= 40000:
        wu = -w.flip(0, 1)
        b = compress(cbk, wu)
        ref.assert_within(cbk.ffn_gated(a, b, x.cuda()), *ref.ffn("silu", x, w, wu), "ffn_gated")
        for name, g, r in zip(("dX", "dG", "dU"), cbk.ffn_gated_bwd(a, b, x.cuda(), dy.cuda()), ref.ffn_bwd("silu", x, w, wu, dy)):
            ref.assert_within(g, *r, name)


def test_a_leading_dimension_past_the_fast_kernels(env):
    torch, cbk = env
    w = weights(torch, 50, 64, 700, 56, 0.1)
    for T in (3, 300):
        x = acts(torch, T, 64, 57)
        big = torch.zeros(T, (1 << 21) + 8, dtype=torch.bfloat16, device="cuda")[:, :64]
        big.copy_(x)
        ref.assert_within(cbk.linear(compress(cbk, w), big), *ref.linear(x, w), "linear")


@pytest.mark.parametrize("T", [1, 20, 400])
def test_corrupt_indices_read_as_nan(env, T):
    """Indices at or past U name 0x7FC0; every way of decoding agrees with cbk_decode_bf16."""
    torch, cbk = env
    rows, cols, U = 70, 192, 300  # b = 9, 212 of 512 indices corrupt
    g = torch.Generator().manual_seed(58)
    words = torch.randint(-(1 << 31), 1 << 31, (cbk.words_for(rows * cols, 9),), generator=g).int().cuda()
    codebook = torch.arange(16000, 16000 + U).short().cuda()
    for c in (cols, 191):
        t = cbk.Compressed(rows, c, U, 9, codebook, words)
        w = cbk.decode_bf16(t).cpu()
        x = acts(torch, T, c, 59)
        y = cbk.linear(t, x.cuda()).cpu()
        assert torch.equal(torch.isnan(y), torch.isnan(x.float() @ w.float().T))
        sparse = cbk.Compressed(rows, c, U, 9, codebook, torch.where(torch.rand(words.shape, generator=g).cuda() < 0.995, 0, words))
        w = cbk.decode_bf16(sparse).cpu()
        assert bool(torch.isnan(w).any()) and not bool(torch.isnan(w).all(1).any())
        clean = torch.isnan(w).any(1).logical_not()
        y = cbk.linear(sparse, x.cuda()).cpu()
        assert bool(torch.isnan(y[:, ~clean]).all())
        ref.assert_within(y[:, clean], *ref.linear(x, w[clean]), "clean rows")


@pytest.mark.parametrize("T", [1, 20, 300, 700])
def test_captured_graphs(env, T):
    """Two captured calls with workspaces of their own, replayed in turn several times with new inputs
    and eager work in between."""
    torch, cbk = env
    rows, cols = 320, 192
    wg, wu = weights(torch, rows, cols, 1500, 60, 0.2), -weights(torch, rows, cols, 1500, 60, 0.2).flip(0, 1)
    a, b = compress(cbk, wg), compress(cbk, wu)
    X, dH = torch.empty(T, cols, dtype=torch.bfloat16, device="cuda"), torch.empty(T, rows, dtype=torch.bfloat16, device="cuda")
    labels = torch.zeros(T, dtype=torch.int64, device="cuda")
    dloss = torch.ones(T, device="cuda")

    def block():
        return list(cbk.ffn_gated_bwd(a, b, X, dH)) + [cbk.ffn_gated(a, b, X), cbk.linear(a, X), cbk.linear_dx(a, dH)]

    def head():
        loss, lse = cbk.xent(a, X, labels)
        return [loss, lse, cbk.xent_bwd(a, X, labels, lse, dloss)]

    graphs = []
    for f in (block, head):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = f()
        graphs.append((g, outs, f))
    for i in range(4):
        X.copy_(acts(torch, T, cols, 61 + i))
        dH.copy_(acts(torch, T, rows, 71 + i, 0.1))
        labels.copy_(torch.randint(0, rows, (T,), generator=torch.Generator().manual_seed(81 + i)))
        for g, outs, f in graphs:
            g.replay()
            want = f()
            torch.cuda.synchronize()
            for got, w in zip(outs, want):
                assert torch.equal(bits(torch, got), bits(torch, w)), i


def test_other_streams_and_a_given_workspace(env):
    torch, cbk = env
    T, rows, cols = 40, 500, 256
    w = weights(torch, rows, cols, 1500, 62, 0.2)
    a = compress(cbk, w)
    xs = [acts(torch, T, cols, 63 + i).cuda() for i in range(4)]
    want = [cbk.linear(a, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    need = cbk.linear_workspace_bytes(a, T)
    spaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    given = [cbk.linear(a, x, stream=s, workspace=ws) for x, s, ws in zip(xs, streams, spaces)]
    own = [cbk.linear(a, x, stream=s) for x, s in zip(xs, streams)]
    inside = []
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            inside.append(cbk.linear(a, x))
    torch.cuda.synchronize()
    for group in (given, own, inside):
        for got, w in zip(group, want):
            assert torch.equal(bits(torch, got), bits(torch, w))
    with pytest.raises(cbk.CbkError) as e:
        cbk.linear(a, xs[0], workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 2
    with pytest.raises(cbk.CbkError) as e:
        cbk.linear(a, xs[0], workspace=torch.empty(need + 256, dtype=torch.uint8, device="cuda")[1:])
    assert e.value.status == 3
    with pytest.raises(ValueError, match="are on"):
        cbk.linear(a, xs[0], out=torch.empty(T, rows, dtype=torch.bfloat16))


def test_words_past_4_gb(env):
    """2.7 billion weights of 13 bits: 4.4 GB of index words, the last rows checked on their own."""
    torch, cbk = env
    rows, cols, T = 330_000, 8192, 3
    g = torch.Generator(device="cuda").manual_seed(64)
    w = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 30_000):
        w[r: r + 30_000] = (torch.randn(min(30_000, rows - r), cols, generator=g, device="cuda") * 0.02).bfloat16()
    t = cbk.encode_gpu(w)
    assert t.b == 13 and t.words.numel() * 4 > 1 << 32
    last = w[-500:].cpu()
    x, dy = acts(torch, T, cols, 65), torch.zeros(T, rows, dtype=torch.bfloat16)
    dy[:, -500:] = acts(torch, T, 500, 66)
    del w
    for n in (1, T):
        y = cbk.linear(t, x[:n].cuda())
        ref.assert_within(y[:, -500:], *ref.linear(x[:n], last), "linear")
        dx = cbk.linear_dx(t, dy[:n].cuda())
        want, bound = ref.linear_dx(dy[:n, -500:], last)
        ref.assert_within(dx, want, bound, "linear_dx")
    X = acts(torch, 400, cols, 67)
    y = cbk.linear(t, X.cuda())  # decoded first, a piece at a time
    ref.assert_within(y[:, -500:], *ref.linear(X, last), "linear, pieces")


@pytest.mark.parametrize("T", [1, 37, 400])
def test_a_block_and_a_head_together(env, T):
    """x -> gated block -> down projection -> head's loss, and back to x: each step's result against the
    reference on the inputs that it was given, so every step's own bound holds, and the whole chain's
    gradient against float64 autograd."""
    torch, cbk = env
    K, F, V = 192, 640, 1000
    wg, wu, wd, wv = (weights(torch, *s, 2000, 90 + i, 0.08) for i, s in enumerate(((F, K), (F, K), (K, F), (V, K))))
    g, u, d, v = (compress(cbk, w) for w in (wg, wu, wd, wv))
    x = acts(torch, T, K, 95)
    gen = torch.Generator().manual_seed(96)
    labels = torch.randint(0, V, (T,), generator=gen)
    labels[1::6] = -100
    weight = (torch.rand(T, generator=gen) + 0.5) / T
    xd, ld, wt = x.cuda(), labels.cuda(), weight.cuda()

    h = cbk.ffn_gated(g, u, xd)
    y = cbk.linear(d, h)
    loss, lse = cbk.xent(v, y, ld)
    dy = cbk.xent_bwd(v, y, ld, lse, wt)
    dh = cbk.linear_dx(d, dy)
    dx, dg, du = cbk.ffn_gated_bwd(g, u, xd, dh)

    hc, yc, dyc, dhc = (t.cpu() for t in (h, y, dy, dh))
    ref.assert_within(h, *ref.ffn("silu", x, wg, wu), "h")
    ref.assert_within(y, *ref.linear(hc, wd), "y")
    ref.assert_within(loss, *ref.xent(yc, wv, labels, -100)[0], "loss")
    ref.assert_within(dy, *ref.xent_bwd(yc, wv, labels, weight, -100), "dy")
    ref.assert_within(dh, *ref.linear_dx(dyc, wd), "dh")
    for name, got, want in zip(("dx", "dg", "du"), (dx, dg, du), ref.ffn_bwd("silu", x, wg, wu, dhc)):
        ref.assert_within(got, *want, name)

    z = x.double().requires_grad_()
    a = torch.nn.functional.silu(z @ wg.double().T) * (z @ wu.double().T)
    logits = a @ wd.double().T @ wv.double().T
    per = torch.nn.functional.cross_entropy(logits, labels, reduction="none", ignore_index=-100)
    (per * weight.double()).sum().backward()
    # five BF16 roundings in a row (h, y, dz, dy, dh and dg, du), each of at most 2^-8 and independent in sign:
    # the norm of the whole stays within their sum, doubled for what the products of rounded factors add
    off = (dx.double().cpu() - z.grad).norm() / z.grad.norm()
    assert float(off) <= 2 * 6 * ref.U16, float(off)
    assert float((loss.double().cpu() - per.detach()).abs().max()) <= 2 * 2 * ref.U16 * float(logits.detach().abs().max())


def test_the_loss_changes_as_its_gradient_says(env):
    """Central differences along a direction that BF16 holds exactly: loss(x + d) - loss(x - d) = 2 <g, d>
    up to the third-order term, at most (2 max|dz|)^3 / 3 a token, and the roundings."""
    torch, cbk = env
    T, V, K = 24, 700, 128
    w = weights(torch, V, K, 900, 97, 0.05)
    a = compress(cbk, w)
    gen = torch.Generator().manual_seed(98)
    x = (torch.randint(-16, 17, (T, K), generator=gen) / 16).bfloat16()
    d = (torch.randint(0, 2, (T, K), generator=gen) * 2 - 1).bfloat16() / 64
    assert bool(((x + d).double() == x.double() + d.double()).all())
    labels = torch.randint(0, V, (T,), generator=gen)
    lp, lm = (cbk.xent(a, (x + s * d).cuda(), labels.cuda())[0].double().cpu() for s in (1, -1))
    _, lse = cbk.xent(a, x.cuda(), labels.cuda())
    g = cbk.xent_bwd(a, x.cuda(), labels.cuda(), lse, torch.ones(T).cuda()).double().cpu()
    dz = (d.double() @ w.double().T).abs().amax(1)
    bound = (2 * dz) ** 3 / 3
    for s in (1, -1):
        bound = bound + ref.xent(x + s * d, w, labels, -100)[0][1]
    bound = bound + 2 * (ref.xent_bwd(x, w, labels, torch.ones(T), -100)[1] * d.double().abs()).sum(1)
    off = (lp - lm - 2 * (g * d.double()).sum(1)).abs()
    assert bool((off <= bound).all()), (off - bound).max()
    assert float((lp - lm).abs().max()) > 10 * float(bound.max())  # the test can tell a wrong gradient


@pytest.mark.parametrize("T", [17, 40, 64, 65, 100, 128])
def test_width_8_and_ragged_rows(env, T):
    """Long runs of slices whose fields start anywhere in a dword, at the width with the fewest of them."""
    torch, cbk = env
    rows, cols = 1500, 2001
    w, x = weights(torch, rows, cols, 200, 91), acts(torch, T, cols, 92)
    d = compress(cbk, w)
    assert d.b == 8
    ref.assert_within(cbk.linear(d, x.cuda()), *ref.linear(x, w), "linear")


@pytest.mark.parametrize("T", [1, 30, 500])
def test_one_tensor_as_gate_and_up(env, T):
    torch, cbk = env
    rows, cols = 300, 192
    w, x, dh = weights(torch, rows, cols, 900, 93, 0.2), acts(torch, T, cols, 94), acts(torch, T, rows, 95, 0.1)
    d = compress(cbk, w)
    ref.assert_within(cbk.ffn_gated(d, d, x.cuda()), *ref.ffn("silu", x, w, w), "ffn_gated")
    for name, v, want in zip(("dX", "dG", "dU"), cbk.ffn_gated_bwd(d, d, x.cuda(), dh.cuda()), ref.ffn_bwd("silu", x, w, w, dh)):
        ref.assert_within(v, *want, name)


@pytest.mark.parametrize("T", [1, 2, 16, 45, 200, 300, 384, 500])
@pytest.mark.parametrize("rows,cols,U,V", [(515, 1088, 3000, 700), (300, 1027, 200, 9000)])
def test_pairs_of_two_widths(env, T, rows, cols, U, V):
    torch, cbk = env
    wg, wu = weights(torch, rows, cols, U, 96, 0.1), weights(torch, rows, cols, V, 97, 0.1)
    x, dh = acts(torch, T, cols, 98), acts(torch, T, rows, 99, 0.1)
    g, u = compress(cbk, wg), compress(cbk, wu)
    assert g.b != u.b and min(g.b, u.b) >= 8 and max(g.b, u.b) <= 14
    ref.assert_within(cbk.ffn_gated(g, u, x.cuda()), *ref.ffn("silu", x, wg, wu), "ffn_gated")
    for name, v, want in zip(("dX", "dG", "dU"), cbk.ffn_gated_bwd(g, u, x.cuda(), dh.cuda()), ref.ffn_bwd("silu", x, wg, wu, dh)):
        ref.assert_within(v, *want, name)
