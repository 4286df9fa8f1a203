"""CPU tests of the operators' C ABI (include/cbk_nn.h) and binding: arguments are refused before any
HIP call, no-ops return without one, and workspace sizes follow the documented rules (no GPU is
needed here)."""
import ctypes
import os

import numpy as np
import pytest

OK, INVALID, CAPACITY, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 4
A = 0x10000          # an aligned address that no refused call touches
BIG = 1 << 40        # more workspace than any call here asks for


@pytest.fixture(scope="module")
def cbk():
    import fly_decode_amd
    if not os.path.exists(fly_decode_amd.library_path()):
        from fly_decode_amd import build
        build.build()
    fly_decode_amd.load_library()
    return fly_decode_amd


def tensor(cbk, rows=256, cols=128, U=300, codebook=A, words=A, b=None):
    return cbk._Tensor(rows, cols, U, cbk.bits_for(U) if b is None else b, codebook, words)


def ref(t):
    return ctypes.byref(t) if t is not None else None


class Calls:
    """Each operator with arguments that would be accepted, any of them replaced by name."""

    def __init__(self, cbk):
        self.cbk, self.lib = cbk, cbk.load_library()

    def linear(self, t=None, X=A, ldx=128, T=4, Y=A, ldy=256, ws=A, n=BIG):
        return self.lib.cbk_linear(ref(t or tensor(self.cbk)), X, ldx, T, Y, ldy, ws, n, None)

    def linear_dx(self, t=None, X=A, ldx=256, T=4, Y=A, ldy=128, ws=A, n=BIG):
        return self.lib.cbk_linear_dx(ref(t or tensor(self.cbk)), X, ldx, T, Y, ldy, ws, n, None)

    def ffn(self, t=None, u=None, act=0, X=A, ldx=128, T=4, Y=A, ldy=256, ws=A, n=BIG):
        return self.lib.cbk_ffn_gated(ref(t or tensor(self.cbk)), ref(u or tensor(self.cbk)), act, X, ldx, T, Y, ldy, ws, n, None)

    def ffn_bwd(self, t=None, u=None, act=0, X=A, ldx=128, H=A, ldh=256, T=4, Y=A, ldy=128, G=A, U=A, ldg=256, ws=A, n=BIG):
        return self.lib.cbk_ffn_gated_bwd(ref(t or tensor(self.cbk)), ref(u or tensor(self.cbk)), act, X, ldx, H, ldh, T, Y, ldy,
                                          G, U, ldg, ws, n, None)

    def xent(self, t=None, X=A, ldx=128, L=A, T=4, loss=A, lse=A, ws=A, n=BIG):
        return self.lib.cbk_xent(ref(t or tensor(self.cbk)), X, ldx, L, T, -100, loss, lse, ws, n, None)

    def xent_bwd(self, t=None, X=A, ldx=128, L=A, lse=A, dl=A, T=4, Y=A, ldy=128, ws=A, n=BIG):
        return self.lib.cbk_xent_bwd(ref(t or tensor(self.cbk)), X, ldx, L, lse, dl, T, -100, Y, ldy, ws, n, None)


ALL = ["linear", "linear_dx", "ffn", "ffn_bwd", "xent", "xent_bwd"]


@pytest.mark.parametrize("op", ALL)
def test_refusals_common(cbk, op):
    call = getattr(Calls(cbk), op)
    assert call(X=None) == INVALID
    assert call(X=A + 1) == ALIGN
    assert call(ldx=127) == INVALID
    assert call(ldx=1 << 32) == UNSUPPORTED
    assert call(ws=None) == INVALID
    assert call(ws=A + 128) == ALIGN
    assert call(n=255) == CAPACITY
    assert call(T=1 << 31) == UNSUPPORTED
    assert call(t=tensor(cbk, U=70000, b=17)) == INVALID
    assert call(t=tensor(cbk, b=8)) == INVALID
    assert call(t=tensor(cbk, codebook=None)) == INVALID
    assert call(t=tensor(cbk, words=None)) == INVALID
    assert call(t=tensor(cbk, words=A + 8)) == ALIGN
    assert call(T=0) == OK and call(T=0, X=None, ws=None, n=0) == OK


@pytest.mark.parametrize("op", ["linear", "linear_dx", "ffn", "ffn_bwd", "xent_bwd"])
def test_refusals_output_matrix(cbk, op):
    call = getattr(Calls(cbk), op)
    assert call(Y=None) == INVALID
    assert call(Y=A + 1) == ALIGN
    assert call(ldy=127) == INVALID
    assert call(ldy=1 << 33) == UNSUPPORTED


@pytest.mark.parametrize("op", ["linear", "linear_dx", "xent", "xent_bwd"])
def test_too_wide_or_tall(cbk, op):
    call = getattr(Calls(cbk), op)
    assert call(t=tensor(cbk, rows=1, cols=(1 << 20) + 1), ldx=1 << 21) == UNSUPPORTED
    assert call(t=tensor(cbk, rows=1 << 31, cols=1), ldx=1 << 31) == UNSUPPORTED


@pytest.mark.parametrize("op", ["ffn", "ffn_bwd"])
def test_refusals_pair(cbk, op):
    call = getattr(Calls(cbk), op)
    assert call(act=3) == INVALID and call(act=-1) == INVALID
    assert call(u=tensor(cbk, rows=255)) == INVALID
    assert call(u=tensor(cbk, cols=64)) == INVALID
    assert call(u=tensor(cbk, codebook=None)) == INVALID


def test_refusals_ffn_bwd(cbk):
    call = Calls(cbk).ffn_bwd
    assert call(H=None) == INVALID and call(H=A + 1) == ALIGN and call(ldh=255) == INVALID
    assert call(G=A + 1) == ALIGN and call(U=A + 1) == ALIGN and call(ldg=255) == INVALID
    assert call(G=None, U=None, ldg=0, n=0) == CAPACITY  # both may be left out; the next check is reached


@pytest.mark.parametrize("op", ["xent", "xent_bwd"])
def test_refusals_xent(cbk, op):
    call = getattr(Calls(cbk), op)
    assert call(t=tensor(cbk, rows=0, U=0, codebook=None, words=None)) == INVALID
    assert call(L=None) == INVALID and call(L=A + 4) == ALIGN
    assert call(lse=None) == INVALID and call(lse=A + 2) == ALIGN
    extra = "loss" if op == "xent" else "dl"
    assert call(**{extra: None}) == INVALID and call(**{extra: A + 2}) == ALIGN


def test_workspace_sizes(cbk):
    lib = cbk.load_library()
    t = tensor(cbk, rows=4096, cols=4096, U=5000)
    one = lambda T: lib.cbk_linear_workspace_bytes(ref(t), T)  # noqa: E731
    pair = lambda T: lib.cbk_ffn_workspace_bytes(ref(t), ref(t), T)  # noqa: E731
    head = lambda T: lib.cbk_xent_workspace_bytes(ref(t), T)  # noqa: E731
    for size in (one, pair, head):
        assert size(0) == 0 and size(1 << 31) == 0
        assert 0 < size(1) < (1 << 27)
        # past a chunk of tokens nothing grows
        assert size(8192) == size(100000)
        assert all(size(T) % 256 == 0 for T in (1, 17, 300, 5000))
    assert lib.cbk_linear_workspace_bytes(None, 4) == 0
    assert lib.cbk_ffn_workspace_bytes(ref(t), ref(tensor(cbk, rows=4096, cols=64)), 4) == 0
    # a piece of a large tensor is decoded at a time: far below its 16 GB
    big = tensor(cbk, rows=1 << 20, cols=8192, U=5000)
    assert lib.cbk_linear_workspace_bytes(ref(big), 512) < 1 << 30
    # at few tokens no decoded copy of anything
    assert lib.cbk_linear_workspace_bytes(ref(big), 1) < 64 << 20


def test_python_refuses_before_the_library(cbk):
    torch = pytest.importorskip("torch")
    c = cbk.encode(np.arange(64 * 8, dtype=np.uint16).reshape(8, 64))
    c = cbk.Compressed(c.rows, c.cols, c.U, c.b, torch.from_numpy(c.codebook.view(np.int16)), torch.from_numpy(c.words.view(np.int32)))
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        cbk.linear(c, x)
    with pytest.raises(ValueError, match="X must be"):
        cbk.linear(c, x.float())
    with pytest.raises(ValueError, match="X must be"):
        cbk.linear(c, x[:, :63])
    with pytest.raises(ValueError, match="X must be"):
        cbk.ffn_gated(c, c, torch.zeros(64, 3, dtype=torch.bfloat16).T)
    with pytest.raises(ValueError, match="overlap"):
        cbk.linear(c, x[:1].expand(3, 64))
    with pytest.raises(ValueError, match="act"):
        cbk.ffn_gated(c, c, x, act="relu")
    with pytest.raises(ValueError, match="labels"):
        cbk.xent(c, x, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="labels"):
        cbk.xent(c, x, torch.zeros(6, dtype=torch.int64)[::2])
    with pytest.raises(ValueError, match="dloss"):
        cbk.xent_bwd(c, x, torch.zeros(3, dtype=torch.int64), torch.zeros(3), torch.zeros(4))
    with pytest.raises(ValueError, match="tokens"):
        cbk.ffn_gated_bwd(c, c, x, torch.zeros(2, 8, dtype=torch.bfloat16))
