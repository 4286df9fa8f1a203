"""GPU tests of what the operators in include/cbk_moe.h promise at their edges: captured graphs, streams, workspaces, views
and padding, masked and broken values, corrupt indices, chunks, every width in every size of tile, and a step of a model
from the router to the drawn token and back."""
import ctypes
import math

import pytest

import moe_reference as moe
import nn_reference as ref
from test_gpu_moe import Block, routing
from test_gpu_nn import acts, compress, weights
from test_gpu_nn_edges import bits
from test_gpu_nn_outputs import View
from test_gpu_nn_streams import delay
from test_gpu_nn_workspace import GUARD

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


# (tokens, experts, k, rows, cols, out, patterns): each size of tile, one token unsorted, padded and whole rows, shares of
# a reduction
WAYS = [(1, 4, 2, 128, 192, 64, [900]), (1, 4, 2, 130, 190, 70, [900, 4000]), (12, 4, 2, 128, 192, 64, [900]), (13, 4, 2, 130, 191, 71, [900, 4000]),
        (40, 3, 2, 128, 192, 128, [40000]), (100, 3, 2, 1100, 192, 70, [900]), (200, 2, 2, 130, 191, 320, [9000])]


def same(torch, got, want, what=""):
    for g, w in zip(got, want):
        assert torch.equal(bits(torch, g), bits(torch, w)), what


@pytest.mark.parametrize("T,E,k,rows,cols,out,patterns", WAYS)
def test_captured_graphs(env, T, E, k, rows, cols, out, patterns):
    """Two captured calls, replayed in turn several times with new inputs and eager work in between, against eager calls."""
    torch, cbk = env
    b = Block(torch, cbk, E, rows, cols, out, patterns)
    Z = torch.empty(T, E, device="cuda")
    X, dY = (torch.empty(T, n, dtype=torch.bfloat16, device="cuda") for n in (cols, out))

    def forward():
        e, w = cbk.route(Z, min(k, E), score="sigmoid")
        return [w, cbk.ffn_experts(b.ex, X, e, w)]

    def backward():
        e, w = cbk.route(Z, min(k, E), score="sigmoid")
        dx, dw = cbk.ffn_experts_bwd(b.ex, X, e, w, dY)
        return [dx, dw, cbk.route_bwd(Z, e, dw, score="sigmoid")]

    graphs = []
    for f in (forward, backward):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = f()
        graphs.append((g, outs, f))
    for i in range(4):
        # in turn spread over the experts, and all tokens with the same ones
        Z.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(301 + i)) + (5.0 * torch.arange(E) if i % 2 else 0.0))
        X.copy_(acts(torch, T, cols, 311 + i))
        dY.copy_(acts(torch, T, out, 321 + i, 0.1))
        for g, outs, f in graphs:
            g.replay()
            want = f()
            torch.cuda.synchronize()
            same(torch, outs, want, i)


@pytest.mark.parametrize("T,E,k,rows,cols,out,patterns", WAYS)
def test_streams_beside_pending_work(env, T, E, k, rows, cols, out, patterns):
    """Calls on another stream while others wait on the current one, and an output freed with its use still to run."""
    torch, cbk = env
    b = Block(torch, cbk, E, rows, cols, out, patterns)
    x, dy = [acts(torch, T, cols, 331 + i).cuda() for i in range(2)], acts(torch, T, out, 333, 0.1).cuda()
    e, w = (t.cuda() for t in routing(torch, T, E, k, 334))
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(335)).cuda()

    def run(i, s=None):
        y = cbk.ffn_experts(b.ex, x[i], e, w, stream=s)
        dx, dw = cbk.ffn_experts_bwd(b.ex, x[i], e, w, dy, stream=s)
        return [y, dx, dw, cbk.route(z, 1, stream=s)[1], cbk.route_bwd(z, e, dw, stream=s)]

    want = [run(0), run(1)]
    big = torch.ones(1 << 28, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(2):
        delay(torch, big)
        got.append((run(0), run(1, s)))
    torch.cuda.synchronize()
    for a, c in got:
        same(torch, a, want[0], "current stream")
        same(torch, c, want[1], "other stream")
    y = cbk.ffn_experts(b.ex, x[0], e, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    delay(torch, big)
    copy = y.clone()
    del y
    later = [cbk.ffn_experts(b.ex, x[1], e, w, stream=s) for _ in range(3)]
    torch.cuda.synchronize()
    same(torch, [copy, *later], [want[0][0]] + 3 * [want[1][0]])


@pytest.mark.parametrize("T,E,k,rows,cols,out,patterns", WAYS)
def test_workspace(env, T, E, k, rows, cols, out, patterns):
    """What it holds on entry does not matter, nothing past its bytes is written, and one byte less is refused."""
    torch, cbk = env
    b = Block(torch, cbk, E, rows, cols, out, patterns)
    x, dy = acts(torch, T, cols, 341).cuda(), acts(torch, T, out, 342, 0.1).cuda()
    e, w = (t.cuda() for t in routing(torch, T, E, k, 343))
    calls = {False: lambda ws: [cbk.ffn_experts(b.ex, x, e, w, workspace=ws)],
             True: lambda ws: list(cbk.ffn_experts_bwd(b.ex, x, e, w, dy, workspace=ws))}
    for backward, call in calls.items():
        need = cbk.experts_workspace_bytes(b.ex, T, e.shape[1], backward)
        whole = torch.empty(GUARD + need + GUARD, dtype=torch.uint8, device="cuda")
        results = []
        for fill in (0xFF, 0x00, 0x7F):
            whole.fill_(fill)
            results.append(call(whole[GUARD: GUARD + need]))
            assert bool((whole[:GUARD] == fill).all()) and bool((whole[GUARD + need:] == fill).all()), (backward, fill)
        same(torch, results[1], results[0])
        same(torch, results[2], results[0])
        assert all(bool(torch.isfinite(t).all()) for t in results[0])
        with pytest.raises(cbk.CbkError):
            call(whole[GUARD: GUARD + need - 1])


@pytest.mark.parametrize("T,E,k,rows,cols,out,patterns", WAYS)
def test_views(env, T, E, k, rows, cols, out, patterns):
    """Rows with padding, from any element: the same bits as whole ones, nothing read of what surrounds inputs, nothing
    written beside outputs."""
    torch, cbk = env
    lib = cbk.load_library()
    b = Block(torch, cbk, E, rows, cols, out, patterns)
    x, dy = acts(torch, T, cols, 351), acts(torch, T, out, 352, 0.1)
    e, w = routing(torch, T, E, k, 353)
    e, w, n = e.cuda(), w.cuda(), e.shape[1]
    want = [cbk.ffn_experts(b.ex, x.cuda(), e, w), *cbk.ffn_experts_bwd(b.ex, x.cuda(), e, w, dy.cuda())]
    stream = torch.cuda.current_stream().cuda_stream
    for pad, lead in (((-cols) % 8, 0), (4, 4), (8, 1), (5, 3)):
        vx, vdy, y, dx = (View(torch, T, m, pad, lead) for m in (cols, out, out, cols))
        for v, values in ((vx, x), (vdy, dy)):
            v.whole.fill_(math.nan)
            v.x.copy_(values)
        guarded = [torch.full((T * n + 8,), 7.0, device="cuda") for _ in range(2)]
        ex = ctypes.byref(b.ex._struct)
        for backward in (0, 1):
            need = lib.cbk_experts_workspace_bytes(ex, T, n, backward)
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            if backward:
                st = lib.cbk_ffn_experts_bwd(ex, 0, vx.ptr(), vx.ld, T, e.data_ptr(), w.data_ptr(), n, vdy.ptr(), vdy.ld, dx.ptr(), dx.ld,
                                             guarded[0][4:].data_ptr(), ws.data_ptr(), need, stream)
            else:
                st = lib.cbk_ffn_experts(ex, 0, vx.ptr(), vx.ld, T, e.data_ptr(), w.data_ptr(), n, y.ptr(), y.ld, ws.data_ptr(), need, stream)
            assert st == 0
        same(torch, [y.x, dx.x, guarded[0][4:-4].view(T, n)], want, (pad, lead))
        assert bool((guarded[0][:4] == 7).all()) and bool((guarded[0][-4:] == 7).all())
        assert y.surroundings_are_as_before() and dx.surroundings_are_as_before()
        # dweights that are not wanted
        need = lib.cbk_experts_workspace_bytes(ex, T, n, 1)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert lib.cbk_ffn_experts_bwd(ex, 0, vx.ptr(), vx.ld, T, e.data_ptr(), w.data_ptr(), n, vdy.ptr(), vdy.ld, dx.ptr(), dx.ld,
                                       None, ws.data_ptr(), need, stream) == 0
        same(torch, [dx.x], want[1:2])


@pytest.mark.parametrize("T", [1, 12, 40, 200])
@pytest.mark.parametrize("patterns", [[900, 3], [15000, 9000], [40000]])
def test_codebooks_from_any_element(env, T, patterns):
    torch, cbk = env
    b = Block(torch, cbk, 3, 200, 257, 210, patterns)
    x, dy = acts(torch, T, 257, 361).cuda(), acts(torch, T, 210, 362, 0.1).cuda()
    e, w = (t.cuda() for t in routing(torch, T, 3, 2, 363))
    moved, n = [], 0
    for ts in b.ex.tensors:
        moved.append([])
        for t in ts:
            n += 1
            at = n % 8
            whole = torch.full((t.codebook.numel() + 16,), 0x7FC0, dtype=t.codebook.dtype, device="cuda")
            whole[at: at + t.codebook.numel()] = t.codebook
            moved[-1].append(cbk.Compressed(t.rows, t.cols, t.U, t.b, whole[at: at + t.codebook.numel()], t.words))
    ex = cbk.Experts(*moved)
    same(torch, [cbk.ffn_experts(ex, x, e, w), *cbk.ffn_experts_bwd(ex, x, e, w, dy)],
         [cbk.ffn_experts(b.ex, x, e, w), *cbk.ffn_experts_bwd(b.ex, x, e, w, dy)])


@pytest.mark.parametrize("T,E,k,rows,cols,out,patterns", WAYS)
def test_unused_slots_and_broken_values(env, T, E, k, rows, cols, out, patterns):
    """Tokens without experts, whatever their rows and weights hold, give and get zeros; the others' results are as
    without them, also where an expert that none of them uses is full of infinities."""
    torch, cbk = env
    b = Block(torch, cbk, E, rows, cols, out, patterns)
    x, dy = acts(torch, T, cols, 371), acts(torch, T, out, 372, 0.1)
    e, w = routing(torch, T, E, k, 373)
    e[e == 1] = 0
    broken = torch.arange(T) % 3 == (0 if T > 1 else 1)
    if T > 3:
        e[T // 2:T // 2 + 2] = torch.tensor([1 << 30, -(1 << 31)][: e.shape[1]] + [E] * (e.shape[1] - 2), dtype=torch.int32)
        broken[T // 2:T // 2 + 2] = True
    e[broken] = torch.where(e[broken] >= 0, -1 - e[broken], e[broken])
    want = [cbk.ffn_experts(b.ex, x.cuda(), e.cuda(), w.cuda()), *cbk.ffn_experts_bwd(b.ex, x.cuda(), e.cuda(), w.cuda(), dy.cuda())]
    bad = [[compress(cbk, torch.where(torch.rand(t.shape) < 0.5, math.inf, math.nan).bfloat16()) if i == 1 else c
            for i, (t, c) in enumerate(zip(ts, cs))] for ts, cs in zip((b.wg, b.wu, b.wd), b.ex.tensors)]
    ex = cbk.Experts(*bad)
    x[broken], dy[broken] = math.nan, math.inf
    w = torch.where((e >= 0) & (e < E), w, math.nan)
    got = [cbk.ffn_experts(ex, x.cuda(), e.cuda(), w.cuda()), *cbk.ffn_experts_bwd(ex, x.cuda(), e.cuda(), w.cuda(), dy.cuda())]
    same(torch, got, want)
    for t in got:
        assert bool((t.cpu()[broken] == 0).all()) and bool(t.isfinite().all())


@pytest.mark.parametrize("T", [1, 9, 40, 200])
def test_no_slots_and_the_same_expert_in_every_slot(env, T):
    torch, cbk = env
    b = Block(torch, cbk, 3, 128, 192, 100, [900])
    x, dy = acts(torch, T, 192, 381), acts(torch, T, 100, 382, 0.1)
    w = torch.rand(T, 4, generator=torch.Generator().manual_seed(383))
    none = torch.full((T, 4), 3, dtype=torch.int32)
    y = cbk.ffn_experts(b.ex, x.cuda(), none.cuda(), w.cuda())
    dx, dw = cbk.ffn_experts_bwd(b.ex, x.cuda(), none.cuda(), w.cuda(), dy.cuda())
    assert all(bool((t == 0).all()) for t in (y, dx, dw))
    e = torch.full((T, 4), 2, dtype=torch.int32)
    y = cbk.ffn_experts(b.ex, x.cuda(), e.cuda(), w.cuda())
    ref.assert_within(y, *moe.experts("silu", b.wg, b.wu, b.wd, x, e, w), "Y")
    got = cbk.ffn_experts_bwd(b.ex, x.cuda(), e.cuda(), w.cuda(), dy.cuda())
    for name, g, want in zip(("dX", "dweights"), got, moe.experts_bwd("silu", b.wg, b.wu, b.wd, x, e, w, dy)):
        ref.assert_within(g, *want, name)


@pytest.mark.parametrize("T", [1, 12, 40, 200])
@pytest.mark.parametrize("cols", [192, 190])
def test_corrupt_indices_read_as_nan(env, T, cols):
    """A corrupt index in a row of gate or up makes a hidden column NaN, in a row of down a column of Y; other experts'
    tokens are as they were."""
    torch, cbk = env
    rows, out, U = 70, 64, 300  # b = 9, 212 of 512 indices corrupt
    b = Block(torch, cbk, 3, rows, cols, out, [U])
    x, dy = acts(torch, T, cols, 391).cuda(), acts(torch, T, out, 392, 0.1).cuda()
    e, w = routing(torch, T, 3, 2, 393, unused=False)
    e[0, 0], e[0, 1] = 1, 0
    hit = (e == 1).any(1)
    w = w.cuda() + 0.1
    want = [cbk.ffn_experts(b.ex, x, e.cuda(), w), *cbk.ffn_experts_bwd(b.ex, x, e.cuda(), w, dy)]

    def broken(kind, row, col):
        t = b.ex.tensors[kind][1]
        words = t.words.clone()
        bit = (row * t.cols + col) * t.b
        mask = ((1 << t.b) - 1) << (bit % 32)  # all ones: index 511
        for i, part in ((bit // 32, mask & 0xFFFFFFFF), (bit // 32 + 1, mask >> 32)):
            if part:
                words[i] |= part - (1 << 32) if part >> 31 else part
        tensors = [list(ts) for ts in b.ex.tensors]
        tensors[kind][1] = cbk.Compressed(t.rows, t.cols, U, t.b, t.codebook, words)
        assert bool(cbk.decode_bf16(tensors[kind][1])[row, col].isnan())
        return cbk.Experts(*tensors)

    assert b.ex.tensors[0][1].b == 9 and b.ex.tensors[2][1].b == 9
    for kind in (0, 1):
        y = cbk.ffn_experts(broken(kind, rows - 1, cols - 1), x, e.cuda(), w)
        assert bool(y[hit.cuda()].isnan().all())
        same(torch, [y.cpu()[~hit]], [want[0].cpu()[~hit]])
        dx, dw = cbk.ffn_experts_bwd(broken(kind, rows - 1, cols - 1), x, e.cuda(), w, dy)
        assert bool(dx[hit.cuda()].isnan().all()) and bool(dw[(e == 1).cuda()].isnan().all())
        same(torch, [dx.cpu()[~hit], dw.cpu()[e != 1]], [want[1].cpu()[~hit], want[2].cpu()[e != 1]])
    y = cbk.ffn_experts(broken(2, 5, rows - 1), x, e.cuda(), w).cpu()
    assert bool(y[hit, 5].isnan().all())
    y[hit, 5] = want[0].cpu()[hit, 5]
    same(torch, [y], [want[0].cpu()])


# tables of 2^13 to 2^16 entries: a pair in LDS or not, down in LDS or not, with each size of tile
@pytest.mark.parametrize("T", [1, 4, 40, 300])
@pytest.mark.parametrize("patterns", [[7000, 7000, 15000], [7000, 15000, 7000], [15000], [20000, 500, 900], [500, 900, 60000], [40000]])
def test_wide_indices(env, T, patterns):
    torch, cbk = env
    rows, cols, out = 260, 300, 270
    wg, wu, wd = (weights(torch, *s, patterns[i % len(patterns)], 401 + i, 0.1) for i, s in enumerate(((rows, cols), (rows, cols), (out, rows))))
    other = [weights(torch, *s, 50, 404 + i, 0.1) for i, s in enumerate(((rows, cols), (rows, cols), (out, rows)))]
    lists = [[a, o] for a, o in zip((wg, wu, wd), other)]
    ex = cbk.Experts(*([compress(cbk, t) for t in ts] for ts in lists))
    x, dy = acts(torch, T, cols, 407), acts(torch, T, out, 408, 0.1)
    e, w = routing(torch, T, 2, 1, 409, unused=False)
    e[0] = 0
    y = cbk.ffn_experts(ex, x.cuda(), e.cuda(), w.cuda())
    ref.assert_within(y, *moe.experts("silu", *lists, x, e, w), "Y")
    got = cbk.ffn_experts_bwd(ex, x.cuda(), e.cuda(), w.cuda(), dy.cuda())
    for name, g, want in zip(("dX", "dweights"), got, moe.experts_bwd("silu", *lists, x, e, w, dy)):
        ref.assert_within(g, *want, name)


@pytest.mark.parametrize("T,k", [(5, 64), (700, 3)])
def test_a_thousand_experts(env, T, k):
    torch, cbk = env
    E = 1024
    made = [[(t, compress(cbk, t)) for t in (weights(torch, r, c, 40, 411 + 10 * j + i, 0.2) for i in range(5))] for j, (r, c) in enumerate(((24, 40), (24, 40), (30, 24)))]
    lists = [[m[i * (j + 1) % 5] for i in range(E)] for j, m in enumerate(made)]
    ex = cbk.Experts(*([c for _, c in ts] for ts in lists))
    x, dy = acts(torch, T, 40, 421), acts(torch, T, 30, 422, 0.1)
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(423))
    e, w = cbk.route(z.cuda(), k)
    want, _ = moe.route(z, k)
    assert torch.equal(e.cpu(), want)
    ws = [[t for t, _ in ts] for ts in lists]
    y = cbk.ffn_experts(ex, x.cuda(), e, w)
    ref.assert_within(y, *moe.experts("silu", *ws, x, want, w.cpu()), "Y")
    got = cbk.ffn_experts_bwd(ex, x.cuda(), e, w, dy.cuda())
    for name, g, r in zip(("dX", "dweights"), got, moe.experts_bwd("silu", *ws, x, want, w.cpu(), dy)):
        ref.assert_within(g, *r, name)


def test_several_chunks_of_tokens(env):
    torch, cbk = env
    T, k = 47000, 3  # 21845 tokens of 3 slots in a chunk
    b = Block(torch, cbk, 2, 64, 64, 40, [60])
    x, dy = acts(torch, T, 64, 431), acts(torch, T, 40, 432, 0.1)
    e, w = routing(torch, T, 2, k, 433)
    assert cbk.experts_workspace_bytes(b.ex, T, k) == cbk.experts_workspace_bytes(b.ex, 10 * T, k)
    y = cbk.ffn_experts(b.ex, x.cuda(), e.cuda(), w.cuda())
    ref.assert_within(y, *moe.experts("silu", b.wg, b.wu, b.wd, x, e, w), "Y")
    got = cbk.ffn_experts_bwd(b.ex, x.cuda(), e.cuda(), w.cuda(), dy.cuda())
    for name, g, want in zip(("dX", "dweights"), got, moe.experts_bwd("silu", b.wg, b.wu, b.wd, x, e, w, dy)):
        ref.assert_within(g, *want, name)


def test_more_tokens_than_a_launch_has_threads_for(env):
    torch, cbk = env
    T = (1 << 26) + 5
    z = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    z[-3:] = -math.inf
    e, w = cbk.route(z, 1)
    assert bool((e[:-3] == 0).all()) and bool((w[:-3] == 1).all()) and bool((e[-3:] == -1).all()) and bool((w[-3:] == 0).all())
    dz = cbk.route_bwd(z, e, w, score="sigmoid", renormalise=False)
    assert bool((dz[:-3] == 0.25).all()) and bool((dz[-3:] == 0).all())


def test_calls_that_are_refused(env):
    torch, cbk = env
    b = Block(torch, cbk, 2, 64, 64, 40, [60])
    x, dy = acts(torch, 5, 64, 441).cuda(), acts(torch, 5, 40, 442).cuda()
    e, w = torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.ones(5, 2, device="cuda")
    z = torch.randn(5, 8, device="cuda")
    for call in (lambda: cbk.ffn_experts(b.ex, x.float(), e, w), lambda: cbk.ffn_experts(b.ex, x[:, :63], e, w), lambda: cbk.ffn_experts(b.ex, x[:4], e, w),
                 lambda: cbk.ffn_experts(b.ex, x, e.long(), w), lambda: cbk.ffn_experts(b.ex, x, e, w.bfloat16()), lambda: cbk.ffn_experts(b.ex, x, e.T.contiguous().T, w),
                 lambda: cbk.ffn_experts(b.ex, x, e, w[:, :1]), lambda: cbk.ffn_experts(b.ex, x, e, w, act="relu"), lambda: cbk.ffn_experts(b.ex, x, e, w, out=x),
                 lambda: cbk.ffn_experts(b.ex, x, e, w.clone().requires_grad_()), lambda: cbk.ffn_experts(b.ex, x.clone().requires_grad_(), e, w),
                 lambda: cbk.ffn_experts(b.ex, x, e.cpu(), w), lambda: cbk.ffn_experts(b.ex, x.cpu(), e.cpu(), w.cpu()),
                 lambda: cbk.ffn_experts_bwd(b.ex, x, e, w, dy[:4]), lambda: cbk.ffn_experts_bwd(b.ex, x, e, w, x), lambda: cbk.ffn_experts_bwd(b.ex, x, e, w, dy, dX=dy),
                 lambda: cbk.ffn_experts_bwd(b.ex, x, e, w, dy.clone().requires_grad_()), lambda: cbk.ffn_experts_bwd(b.ex, x, e, w, dy.expand(5, 40)[:1].expand(5, 40)),
                 lambda: cbk.route(z, 2, bias=torch.zeros(8)), lambda: cbk.route(z, 1 << 40), lambda: cbk.route(z, 2, groups=(1 << 32) + 1),
                 lambda: cbk.route(z.clone().requires_grad_(), 2), lambda: cbk.sample(z, torch.rand(5, device="cuda"), top_k=1 << 40),
                 lambda: cbk.sample(z, torch.rand(5)), lambda: cbk.sample(z, torch.rand(5, device="cuda"), temperature=torch.ones(5))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cbk.route(z, 0), lambda: cbk.route(z, 9), lambda: cbk.route(z, 2, groups=3), lambda: cbk.route(z, 2, groups=2, top_groups=3),
                 lambda: cbk.route(z, 2, group_top=3), lambda: cbk.ffn_experts(b.ex, x, e[:, :0], w[:, :0]),
                 lambda: cbk.ffn_experts(b.ex, x, torch.zeros(5, 65, dtype=torch.int32, device="cuda"), torch.zeros(5, 65, device="cuda"))):
        with pytest.raises(cbk.CbkError):
            call()
    # a table that was made on another device
    elsewhere = cbk.Experts(*b.ex.tensors)
    elsewhere._struct.device = 1
    with pytest.raises(cbk.CbkError):
        cbk.ffn_experts(elsewhere, x, e, w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError):
            cbk.Experts(*b.ex.tensors)
        y = cbk.ffn_experts(b.ex, x, e, w)
    g.replay()
    same(torch, [y], [cbk.ffn_experts(b.ex, x, e, w)])


def test_no_tokens(env):
    torch, cbk = env
    b = Block(torch, cbk, 2, 64, 64, 40, [60])
    x, dy = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    e, w = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    assert cbk.ffn_experts(b.ex, x, e, w).shape == (0, 40)
    dx, dw = cbk.ffn_experts_bwd(b.ex, x, e, w, dy)
    assert dx.shape == (0, 64) and dw.shape == (0, 2)
    z = torch.empty(0, 9, device="cuda")
    assert [tuple(t.shape) for t in cbk.route(z, 4)] == [(0, 4)] * 2 and cbk.route_bwd(z, e, w).shape == (0, 9)
    assert [tuple(t.shape) for t in cbk.sample(z, torch.empty(0, device="cuda"))] == [(0,)] * 2


def test_gradient_against_differences(env):
    """dX and dweights against central differences of the formula in 64 bits."""
    torch, cbk = env
    b = Block(torch, cbk, 3, 20, 12, 10, [50])
    T = 4
    x, dy = acts(torch, T, 12, 451), acts(torch, T, 10, 452)
    e, w = routing(torch, T, 3, 2, 453)
    dx, dw = cbk.ffn_experts_bwd(b.ex, x.cuda(), e.cuda(), w.cuda(), dy.cuda())
    (_, bx), (_, bw) = moe.experts_bwd("silu", b.wg, b.wu, b.wd, x, e, w, dy)

    def value(x64, w64):
        total = 0.0
        for t in range(T):
            for j in range(2):
                i = int(e[t, j])
                if i >= 0:
                    h = ref.act("silu", x64[t] @ b.wg[i].double().T)[0] * (x64[t] @ b.wu[i].double().T)
                    total = total + w64[t, j] * (b.wd[i].double() @ h) @ dy[t].double()
        return float(total)

    # central differences are off by step^2 / 6 of a third derivative (some 10^3 at most: 20 hidden columns, weights
    # below 1) and by 2^-52 of the value over the step: 1e-7 in all
    step = 1e-5
    for base, got, bound, which in ((x.double(), dx, bx, 0), (w.double(), dw, bw, 1)):
        for t in range(T):
            for j in range(base.shape[1]):
                d = torch.zeros_like(base)
                d[t, j] = step
                args = [(base + s * d, w.double()) if which == 0 else (x.double(), base + s * d) for s in (1, -1)]
                slope = (value(*args[0]) - value(*args[1])) / (2 * step)
                assert abs(slope - float(got[t, j])) <= float(bound[t, j]) + 1e-7, (which, t, j)


@pytest.mark.parametrize("T", [1, 24, 300])
def test_a_step_from_the_router_to_the_token_and_back(env, T):
    """A layer as a model has it -- router, experts, head, a drawn token; then the loss' gradient through all of it, in
    torch.autograd functions -- every operator on what the one before gave, against the reference of each; and the whole
    forward step captured and replayed."""
    torch, cbk = env
    E, k, K, F, V = 12, 3, 128, 192, 700
    b = Block(torch, cbk, E, F, K, K, [900, 2000])
    wr, wh = weights(torch, E, K, 600, 461, 0.3), weights(torch, V, K, 3000, 462, 0.3)
    router, head = compress(cbk, wr), compress(cbk, wh)
    X = acts(torch, T, K, 463).cuda()
    u = torch.rand(T, generator=torch.Generator().manual_seed(464)).cuda()

    def step(x):
        z = cbk.linear(router, x)
        e, w = cbk.route(z, k, score="sigmoid", groups=4, top_groups=2, scale=1.5)
        y = cbk.ffn_experts(b.ex, x, e, w)
        logits = cbk.linear(head, y)
        return z, e, w, y, logits, *cbk.sample(logits, u, temperature=0.7, top_k=40, top_p=0.9)

    z, e, w, y, logits, token, logprob = step(X)
    ref.assert_within(z, *ref.linear(X.cpu(), wr), "router")
    we, ww = moe.route(z.cpu(), k, "sigmoid", None, 4, 2, scale=1.5)
    assert torch.equal(e.cpu(), we) and bool(((w.cpu().double() - ww).abs() <= 2.0 ** -24 * 1.001 * ww).all())
    ref.assert_within(y, *moe.experts("silu", b.wg, b.wu, b.wd, X.cpu(), we, w.cpu()), "experts")
    ref.assert_within(logits, *ref.linear(y.cpu(), wh), "head")
    f32 = lambda v: float(torch.tensor(v))
    for t in range(0, T, 7):
        want, lp = moe.sample(logits[t].tolist(), float(u[t]), f32(0.7), 40, f32(0.9))
        assert int(token[t]) == want and abs(float(logprob[t]) - lp) <= 2.0 ** -24 * abs(lp) + 1e-11
    x2 = X.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(x2)
    for i in range(3):
        x2.copy_(acts(torch, T, K, 465 + i))
        g.replay()
        want = step(x2)
        torch.cuda.synchronize()
        same(torch, [o for o in outs if o.dtype != torch.int64], [o for o in want if o.dtype != torch.int64])
        assert torch.equal(outs[5], want[5])

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, t):
            ctx.t = t
            return cbk.linear(t, x)

        @staticmethod
        def backward(ctx, dy):
            return cbk.linear_dx(ctx.t, dy), None

    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, z):
            e, w = cbk.route(z, k, score="sigmoid", groups=4, top_groups=2, scale=1.5)
            ctx.save_for_backward(z, e)
            ctx.mark_non_differentiable(e)
            return e, w

        @staticmethod
        def backward(ctx, _, dw):
            return cbk.route_bwd(*ctx.saved_tensors, dw.contiguous(), score="sigmoid", scale=1.5)

    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, e, w):
            ctx.save_for_backward(x, e, w)
            return cbk.ffn_experts(b.ex, x, e, w)

        @staticmethod
        def backward(ctx, dy):
            dx, dw = cbk.ffn_experts_bwd(b.ex, *ctx.saved_tensors, dy.contiguous())
            return dx, None, dw

    x = X.clone().requires_grad_()
    z2 = Linear.apply(x, router)
    e2, w2 = Route.apply(z2)
    y2 = Experts.apply(x, e2, w2)
    dy = acts(torch, T, K, 468, 0.1).cuda()
    y2.backward(dy)
    same(torch, [z2.detach(), e2, w2.detach(), y2.detach()], [z, e, w, y])

    dxe, dw = cbk.ffn_experts_bwd(b.ex, X, e, w, dy)
    dz = cbk.route_bwd(z, e, dw, score="sigmoid", scale=1.5)
    dxr = cbk.linear_dx(router, dz)
    (rx, bx), (rw, bw) = moe.experts_bwd("silu", b.wg, b.wu, b.wd, X.cpu(), we, w.cpu(), dy.cpu())
    ref.assert_within(dxe, rx, bx, "dX")
    ref.assert_within(dw, rw, bw, "dweights")
    rz, bz = moe.route_bwd(z.cpu(), we, dw.cpu(), "sigmoid", True, 1.5)
    ref.assert_within(dz, rz, ref.rounded(rz, bz), "dlogits")
    ref.assert_within(dxr, *ref.linear_dx(dz.cpu(), wr), "router's dX")
    assert torch.equal(x.grad, dxe + dxr)


def test_rows_past_4_gb(env):
    """Rows that lie more than 2^32 bytes apart, of inputs and outputs, give what they give side by side."""
    torch, cbk = env
    T, ld = 2200, 1 << 20
    b = Block(torch, cbk, 3, 64, 96, 40, [900])
    big = [torch.zeros(T, ld, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x, dy, z = acts(torch, T, 96, 471).cuda(), acts(torch, T, 40, 472, 0.1).cuda(), acts(torch, T, 3, 473).cuda()
    X, dY, Z, Y, dX, dZ = big[0][:, 8:104], big[0][:, 1000:1040], big[0][:, 2000:2003], big[1][:, 16:56], big[1][:, 101:197], big[1][:, 300:303]
    X.copy_(x), dY.copy_(dy), Z.copy_(z)
    e, w = cbk.route(z, 2)
    same(torch, cbk.route(Z, 2), (e, w))
    y = cbk.ffn_experts(b.ex, x, e, w)
    dx, dw = cbk.ffn_experts_bwd(b.ex, x, e, w, dy)
    cbk.ffn_experts(b.ex, X, e, w, out=Y)
    dW = cbk.ffn_experts_bwd(b.ex, X, e, w, dY, dX=dX)[1]
    cbk.route_bwd(Z, e, dw, out=dZ)
    same(torch, [Y, dX, dW, dZ], [y, dx, dw, cbk.route_bwd(z, e, dw)])
    big[1][:, 16:56], big[1][:, 101:197], big[1][:, 300:303] = 0, 0, 0
    assert not bool(big[1].any())
    # drawing: short rows far apart, and long ones
    u = torch.rand(T, generator=torch.Generator().manual_seed(474)).cuda()
    for kw in ({}, {"top_k": 2}):
        got, want = cbk.sample(Z, u, **kw), cbk.sample(z, u, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    big[0].normal_(generator=torch.Generator(device="cuda").manual_seed(475))
    at = torch.tensor([0, 1, 2047, 2048, 2049, T - 1], device="cuda")
    for kw in ({}, {"top_k": 40}, {"top_p": 0.01}):
        got, want = cbk.sample(big[0], u, **kw), cbk.sample(big[0][at], u[at], **kw)
        assert torch.equal(got[0][at], want[0])
        assert bool(((got[1][at] - want[1]).abs() <= 2.0 ** -23 * want[1].abs() + 1e-11).all())  # (long rows' work may be divided)


@pytest.mark.parametrize("T", [1, 12, 40, 70])
def test_tensors_past_4_gb(env, T):
    """Experts whose index streams are longer than 2^32 bytes, against the block and the products of one such tensor."""
    torch, cbk = env
    rows, cols, out, b = 1 << 20, 2752, 48, 13
    g = torch.Generator(device="cuda").manual_seed(481)
    codebook = (0.02 * torch.randn(1 << b, generator=torch.Generator().manual_seed(482))).bfloat16().view(torch.int16).cuda()

    def tensor(r, c):
        words = torch.empty(cbk.words_for(r * c, b), dtype=torch.int32, device="cuda")
        words.view(torch.uint8).random_(0, 256, generator=g)
        return cbk.Compressed(r, c, 1 << b, b, codebook, words)

    gate, up, down = tensor(rows, cols), tensor(rows, cols), tensor(out, rows)
    assert gate.words.numel() * 4 > 1 << 32
    ex = cbk.Experts([gate, up], [up, gate], [down, down])
    x, dy = acts(torch, T, cols, 483).cuda(), acts(torch, T, out, 484, 0.1).cuda()
    e = (torch.arange(T) % 2)[:, None].int().cuda()
    w = torch.full((T, 1), 0.5, device="cuda")
    y = cbk.ffn_experts(ex, x, e, w)
    dx, dw = cbk.ffn_experts_bwd(ex, x, e, w, dy)
    wd = cbk.decode_bf16(down).float()
    for i, (a, c) in enumerate(((gate, up), (up, gate))):
        part = slice(i, None, 2)
        if T <= i:
            continue
        h = cbk.ffn_gated(a, c, x[part].contiguous())
        want = 0.5 * (h.float() @ wd.T)
        # both round H, whose fp32 sums may differ, to BF16, at most a step apart; the weights' signs are random, so that the
        # differences add up to 8 times the root of the sum of their squares hardly ever; Y is rounded once
        off = 8 * 2.0 ** -7 * torch.sqrt((0.5 * h.float()) ** 2 @ (wd ** 2).T) + 2.0 ** -8 * want.abs()
        assert bool(((y[part].float() - want).abs() <= off).all()) and float(want.abs().mean()) > 4 * float(off.mean())
        dh = (0.5 * (dy[part].float() @ wd)).bfloat16()  # (the experts' is not rounded)
        dX, dG, dU = cbk.ffn_gated_bwd(a, c, x[part].contiguous(), dh)
        # dG and dU differ by dH's rounding, their own, and their factors' sums: by two steps at most; a weight is some 0.02
        size = 0.02 * torch.sqrt((dG.float() ** 2).sum(1) + (dU.float() ** 2).sum(1))[:, None]
        assert bool(((dx[part].float() - dX.float()).abs() <= 8 * 2.0 ** -6 * size + 2.0 ** -7 * dX.float().abs()).all())
        assert float(dX.float().abs().mean()) > 0.3 * float(size.mean())
