"""GPU tests of the outputs of cbk_ffn_gated_bwd and cbk_xent as the C ABI offers them: either of dG and dU,
or both, left out; padded and unaligned rows of theirs; and nothing written beside any output."""
import ctypes

import pytest

from test_gpu_nn import acts, compress, weights
from test_gpu_nn_edges import WAYS, bits

pytestmark = pytest.mark.gpu

MORE = [(400, 300, 192, 3000), (385, 520, 1000, 900)]
ACT = {"silu": 0, "gelu_tanh": 2}


@pytest.fixture(scope="module")
def env():
    import torch
    import fly_decode_amd as cbk
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    cbk.load_library()
    return torch, cbk


class View:
    """[T][n] inside a larger buffer of 7s: row padding, and `lead` elements from a 16-byte boundary."""

    def __init__(self, torch, T, n, pad, lead):
        self.torch, self.ld = torch, n + pad
        self.whole = torch.full(((T + 2) * self.ld + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.at = (self.ld + 7) // 8 * 8 + lead
        self.x = self.whole[self.at: self.at + T * self.ld].view(T, self.ld)[:, :n]

    def ptr(self):
        return self.x.data_ptr()

    def surroundings_are_as_before(self):
        self.x.fill_(7.0)
        return bool((self.whole == 7.0).all())


@pytest.mark.parametrize("want_g,want_u", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("T,rows,cols,U", WAYS + MORE)
def test_dg_and_du_as_wanted(env, T, rows, cols, U, want_g, want_u):
    torch, cbk = env
    lib = cbk.load_library()
    g, u = (compress(cbk, weights(torch, rows, cols, U, 161 + i, 0.2)) for i in range(2))
    X, dH = acts(torch, T, cols, 163).cuda(), acts(torch, T, rows, 164, 0.1).cuda()
    need = cbk.ffn_workspace_bytes(g, u, T)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for act in ACT:
        dX, dG, dU = cbk.ffn_gated_bwd(g, u, X, dH, act=act)
        # whole 16-byte pieces; 8-byte ones; rows on 8 bytes from an odd element; everything odd
        for pad, lead in (((-rows) % 8, 0), ((-rows) % 8 + 4, 4), ((-rows) % 8, 3), ((-rows) % 2 + 5, 1)):
            x, a, b = View(torch, T, cols, 3, 1), View(torch, T, rows, pad, lead), View(torch, T, rows, pad, lead)
            st = lib.cbk_ffn_gated_bwd(ctypes.byref(g._struct()), ctypes.byref(u._struct()), ACT[act], X.data_ptr(), cols,
                                       dH.data_ptr(), rows, T, x.ptr(), x.ld, a.ptr() if want_g else None,
                                       b.ptr() if want_u else None, a.ld if want_g or want_u else 0, ws.data_ptr(), need, stream)
            assert st == 0
            for view, want, wanted in ((x, dX, True), (a, dG, want_g), (b, dU, want_u)):
                if wanted:
                    assert torch.equal(bits(torch, view.x), bits(torch, want)), (act, pad, lead)
                assert view.surroundings_are_as_before(), (act, pad, lead)
    dX2, none_g, none_u = cbk.ffn_gated_bwd(g, u, X, dH, act="silu", projections=False)
    assert none_g is None and none_u is None
    assert torch.equal(bits(torch, dX2), bits(torch, cbk.ffn_gated_bwd(g, u, X, dH, act="silu")[0]))


@pytest.mark.parametrize("T,rows,cols,U", WAYS + MORE)
def test_loss_and_lse_leave_their_surroundings(env, T, rows, cols, U):
    torch, cbk = env
    lib = cbk.load_library()
    t = compress(cbk, weights(torch, rows, cols, U, 165, 0.1))
    X = acts(torch, T, cols, 166).cuda()
    labels = torch.randint(0, rows, (T,), generator=torch.Generator().manual_seed(167)).cuda()
    want = cbk.xent(t, X, labels)
    need = cbk.xent_workspace_bytes(t, T)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for lead in (1, 2, 4):
        whole = [torch.full((T + 16,), 7.0, device="cuda") for _ in range(2)]
        loss, lse = (w[lead: lead + T] for w in whole)
        st = lib.cbk_xent(ctypes.byref(t._struct()), X.data_ptr(), cols, labels.data_ptr(), T, -100, loss.data_ptr(),
                          lse.data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for got, w, all_of_it in zip((loss, lse), want, whole):
            assert torch.equal(bits(torch, got), bits(torch, w))
            got.fill_(7.0)
            assert bool((all_of_it == 7.0).all())
