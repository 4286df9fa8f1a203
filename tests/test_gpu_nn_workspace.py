"""GPU tests of the workspace of the operators in include/cbk_nn.h: what it holds on entry does not matter,
and nothing past the bytes that were asked for is written."""
import pytest

from test_gpu_nn import acts, compress
from test_gpu_nn_edges import WAYS, bits
from test_gpu_nn_sizes import of_width

pytestmark = pytest.mark.gpu

# tokens, rows, cols, width of a tensor and of a pair's second: decoded on the way (one launch, one for each
# tensor), decoded first with shared tiles, in pieces, in chunks of tokens, by the generic kernel
CASES = [
    (1, 260, 256, 12, 12), (20, 261, 131, 12, 12), (20, 260, 256, 12, 9), (300, 515, 1088, 13, 13), (256, 515, 1088, 14, 14),
    (100, 300, 1027, 11, 8), (385, 20000, 300, 11, 11), (500, 300, 20000, 12, 12), (2100, 300, 8192, 12, 11),
    (300, 70000, 64, 10, 10), (200, 70000, 64, 10, 10), (8200, 40, 70, 9, 9), (400, 1001, 1001, 15, 3), (30, 70, 128, 5, 0),
]
GUARD = 1 << 16


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


@pytest.mark.parametrize("T,rows,cols,b,second", CASES)
def test_contents_on_entry_and_bytes_past_the_end(env, T, rows, cols, b, second):
    torch, cbk = env

    def tensor(width, seed):
        return of_width(torch, rows, cols, width, seed) if width else torch.full((rows, cols), 0.03125, dtype=torch.bfloat16)

    a, c = compress(cbk, tensor(b, 151)), compress(cbk, tensor(second, 152))
    assert (a.b, c.b) == (b, second)
    X, dY = acts(torch, T, cols, 153).cuda(), acts(torch, T, rows, 154, 0.1).cuda()
    labels = torch.randint(0, rows, (T,), generator=torch.Generator().manual_seed(155)).cuda()
    labels[::7] = -100
    dloss = torch.rand(T, generator=torch.Generator().manual_seed(156)).cuda()
    lse = cbk.xent(a, X, labels)[1]
    calls = {
        "linear": (cbk.linear_workspace_bytes(a, T), lambda ws: [cbk.linear(a, X, workspace=ws)]),
        "linear_dx": (cbk.linear_workspace_bytes(a, T), lambda ws: [cbk.linear_dx(a, dY, workspace=ws)]),
        "ffn_gated": (cbk.ffn_workspace_bytes(a, c, T), lambda ws: [cbk.ffn_gated(a, c, X, workspace=ws)]),
        "ffn_gated_bwd": (cbk.ffn_workspace_bytes(a, c, T), lambda ws: list(cbk.ffn_gated_bwd(a, c, X, dY, workspace=ws))),
        "xent": (cbk.xent_workspace_bytes(a, T), lambda ws: list(cbk.xent(a, X, labels, workspace=ws))),
        "xent_bwd": (cbk.xent_workspace_bytes(a, T), lambda ws: [cbk.xent_bwd(a, X, labels, lse, dloss, workspace=ws)]),
    }
    for name, (need, call) in calls.items():
        whole = torch.empty(GUARD + need + GUARD, dtype=torch.uint8, device="cuda")
        results = []
        for fill in (0xFF, 0x00, 0x7F):
            whole.fill_(fill)
            results.append(call(whole[GUARD: GUARD + need]))
            assert bool((whole[:GUARD] == fill).all()) and bool((whole[GUARD + need:] == fill).all()), (name, fill)
        for other in results[1:]:
            for got, want in zip(other, results[0]):
                assert torch.equal(bits(torch, got), bits(torch, want)), name
        assert all(bool(torch.isfinite(t).all()) for t in results[0]), name


@pytest.mark.parametrize("T,rows,cols,U", WAYS)
def test_one_byte_less_is_refused(env, T, rows, cols, U):
    torch, cbk = env
    a = compress(cbk, of_width(torch, rows, cols, 10, 157))
    X = acts(torch, T, cols, 158).cuda()
    for need, call in ((cbk.linear_workspace_bytes(a, T), cbk.linear), (cbk.ffn_workspace_bytes(a, a, T), lambda t, x, **k: cbk.ffn_gated(t, t, x, **k))):
        with pytest.raises(cbk.CbkError) as e:
            call(a, X, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == 2
