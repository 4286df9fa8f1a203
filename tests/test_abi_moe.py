"""CPU tests of the C ABI and the binding of include/cbk_moe.h and include/cbk_sample.h: arguments are refused before any
HIP call, no-ops return without one, and workspace sizes follow the documented rules (no GPU is needed here)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def router(cbk, **kw):
    return cbk._Router(**{"experts": 16, "k": 4, "score": 0, "renormalise": 1, "scale": 1.0, "groups": 1, "top_groups": 1, "group_top": 1, **kw})


def block(cbk, **kw):
    return cbk._Experts(**{"buffer": A, "rows": 256, "cols": 128, "out": 192, "count": 8, "b": 12, "b_down": 13, "device": 0, **kw})


class Calls:
    """Each call with arguments that would be accepted, any of them replaced by name."""

    def __init__(self, cbk):
        self.cbk, self.lib = cbk, cbk.load_library()

    def route(self, r=None, Z=A, dtype=0, ld=16, T=4, bias=A, E=A, W=A):
        return self.lib.cbk_route(ctypes.byref(r or router(self.cbk)), Z, dtype, ld, T, bias, E, W, None)

    def route_bwd(self, r=None, Z=A, dtype=0, ld=16, T=4, E=A, W=A, Y=A, ldy=16):
        return self.lib.cbk_route_bwd(ctypes.byref(r or router(self.cbk)), Z, dtype, ld, T, E, W, Y, ldy, None)

    def experts(self, ex=None, act=0, Z=A, ld=128, T=4, E=A, W=A, k=2, Y=A, ldy=192, ws=A, n=BIG):
        return self.lib.cbk_ffn_experts(ctypes.byref(ex or block(self.cbk)), act, Z, ld, T, E, W, k, Y, ldy, ws, n, None)

    def experts_bwd(self, ex=None, act=0, Z=A, ld=128, T=4, E=A, W=A, k=2, G=A, ldg=192, Y=A, ldy=128, D=A, ws=A, n=BIG):
        return self.lib.cbk_ffn_experts_bwd(ctypes.byref(ex or block(self.cbk)), act, Z, ld, T, E, W, k, G, ldg, Y, ldy, D, ws, n, None)

    def sample(self, p=None, Z=A, dtype=0, V=16, ld=16, T=4, U=A, Y=A, L=A, ws=A, n=BIG):
        return self.lib.cbk_sample(ctypes.byref(p or self.cbk._Sampling(1.0, 1.0, 0.0, 0)), Z, dtype, ld, V, T, U, Y, L, ws, n, None)


ALL = ["route", "route_bwd", "experts", "experts_bwd", "sample"]


@pytest.mark.parametrize("name", ALL)
def test_no_tokens_is_a_no_op(cbk, name):
    assert getattr(Calls(cbk), name)(T=0, Z=None, **({} if name == "route" else {"Y": None})) == OK


@pytest.mark.parametrize("name", ALL)
def test_too_many_tokens(cbk, name):
    assert getattr(Calls(cbk), name)(T=1 << 31) == UNSUPPORTED


@pytest.mark.parametrize("name,args", [
    ("route", {"Z": None}), ("route", {"E": None}), ("route", {"W": None}), ("route", {"ld": 15}), ("route", {"dtype": 2}),
    ("route_bwd", {"Z": None}), ("route_bwd", {"E": None}), ("route_bwd", {"W": None}), ("route_bwd", {"Y": None}), ("route_bwd", {"ldy": 15}),
    ("experts", {"Z": None}), ("experts", {"E": None}), ("experts", {"W": None}), ("experts", {"Y": None}), ("experts", {"ld": 127}),
    ("experts", {"ldy": 191}), ("experts", {"k": 0}), ("experts", {"act": 3}), ("experts", {"act": -1}), ("experts", {"ws": None}),
    ("experts_bwd", {"Z": None}), ("experts_bwd", {"G": None}), ("experts_bwd", {"Y": None}), ("experts_bwd", {"ldg": 191}),
    ("experts_bwd", {"ldy": 127}), ("experts_bwd", {"k": 0}), ("experts_bwd", {"act": 7}), ("experts_bwd", {"ws": None}),
    ("sample", {"Z": None}), ("sample", {"U": None}), ("sample", {"Y": None}), ("sample", {"V": 0}), ("sample", {"ld": 15}), ("sample", {"dtype": -1}),
    ("sample", {"ws": None}),
])
def test_invalid(cbk, name, args):
    assert getattr(Calls(cbk), name)(**args) == INVALID


@pytest.mark.parametrize("name,args", [
    ("route", {"Z": A + 2}), ("route", {"Z": A + 1, "dtype": 1}), ("route", {"bias": A + 2}), ("route", {"E": A + 2}), ("route", {"W": A + 1}),
    ("route_bwd", {"Y": A + 2}), ("route_bwd", {"W": A + 2}), ("experts", {"Z": A + 1}), ("experts", {"Y": A + 1}), ("experts", {"E": A + 2}),
    ("experts", {"ws": A + 128}), ("experts_bwd", {"D": A + 2}), ("experts_bwd", {"G": A + 1}), ("sample", {"Z": A + 2}), ("sample", {"U": A + 2}),
    ("sample", {"Y": A + 4}), ("sample", {"L": A + 2}), ("sample", {"ws": A + 128}),
])
def test_alignment(cbk, name, args):
    assert getattr(Calls(cbk), name)(**args) == ALIGN


@pytest.mark.parametrize("name,args", [
    ("route", {"ld": 1 << 32}), ("route_bwd", {"ldy": 1 << 32}), ("experts", {"k": 65}), ("experts", {"ld": 1 << 32}),
    ("experts_bwd", {"k": 65}), ("sample", {"V": (1 << 20) + 1, "ld": 1 << 21}), ("sample", {"ld": 1 << 32}),
])
def test_unsupported(cbk, name, args):
    assert getattr(Calls(cbk), name)(**args) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    ({"experts": 0}, INVALID), ({"k": 0}, INVALID), ({"k": 17}, INVALID), ({"score": 2}, INVALID), ({"groups": 0}, INVALID),
    ({"groups": 3}, INVALID), ({"top_groups": 0}, INVALID), ({"top_groups": 2}, INVALID), ({"group_top": 0}, INVALID),
    ({"group_top": 3}, INVALID), ({"experts": 1025}, UNSUPPORTED), ({"experts": 1024, "k": 65}, UNSUPPORTED),
])
def test_routers(cbk, kw, status):
    c = Calls(cbk)
    assert c.route(r=router(cbk, **kw), ld=2000) == status and c.route_bwd(r=router(cbk, **kw), ld=2000, ldy=2000) == status


@pytest.mark.parametrize("kw,status", [
    ({"buffer": None}, INVALID), ({"count": 0}, INVALID), ({"count": 1025}, INVALID), ({"rows": 0}, INVALID), ({"cols": 0}, INVALID),
    ({"out": 0}, INVALID), ({"b": 17}, INVALID), ({"rows": (1 << 20) + 1}, UNSUPPORTED),
])
def test_blocks(cbk, kw, status):
    c = Calls(cbk)
    assert c.experts(ex=block(cbk, **kw)) == status and c.experts_bwd(ex=block(cbk, **kw)) == status
    assert cbk.load_library().cbk_experts_workspace_bytes(ctypes.byref(block(cbk, **kw)), 4, 2, 0) == 0


def test_workspace(cbk):
    lib, c = cbk.load_library(), Calls(cbk)
    ex = block(cbk)
    for backward in (0, 1):
        sizes = [lib.cbk_experts_workspace_bytes(ctypes.byref(ex), T, 2, backward) for T in (0, 1, 100, 5000, 10 ** 6, 10 ** 7, 1 << 31)]
        assert sizes[0] == 0 and sizes[-1] == 0 and sizes[1] <= sizes[2] <= sizes[3] <= sizes[4]
        assert sizes[4] == sizes[5] < 5 << 30  # chunks
        call = c.experts_bwd if backward else c.experts
        assert call(T=100, n=sizes[2] - 1) == CAPACITY
    for k in (0, 65):
        assert lib.cbk_experts_workspace_bytes(ctypes.byref(ex), 4, k, 0) == 0
    # the widest blocks, and many experts: a chunk of one token at least
    wide = block(cbk, rows=1 << 20, cols=1 << 20, out=1 << 20, count=1024)
    assert 0 < lib.cbk_experts_workspace_bytes(ctypes.byref(wide), 1 << 20, 64, 1) < 64 << 30


def test_workspace_of_a_draw(cbk):
    """None for short or many rows with filters; without, chunks of rows."""
    size = cbk.sample_workspace_bytes
    assert size(0, 5) == 0 and size(5, 0) == 0 and size(5, (1 << 20) + 1) == 0 and size(1 << 31, 5) == 0
    assert 0 < size(1, 1) < size(2, 1) and size(1, 1 << 20) < 1 << 20 and size(10 ** 6, 50000) == size(10 ** 5, 50000) <= 64 << 20
    for kw in ({"top_k": 5}, {"top_p": 0.9}, {"min_p": 0.1}):
        assert size(4, 100, **kw) == 0
        assert 32768 < size(1, 100000, **kw) < size(2, 100000, **kw) < size(64, 1 << 20, **kw) < 8 << 20
        assert size(65, 100000, **kw) == 0
    for kw in ({"top_k": 100}, {"top_k": -1}, {"top_p": float("nan")}, {"min_p": -1.0}, {"min_p": float("nan")}):
        assert size(4, 100, **kw) == size(4, 100)
    c = Calls(cbk)
    assert c.sample(n=size(4, 16) - 1) == CAPACITY
    with_filter = cbk._Sampling(1.0, 0.5, 0.0, 0)
    assert c.sample(p=with_filter, ws=None, n=0, U=None) == INVALID  # (U, not the workspace)
    for name in ("temperatures", "top_ps", "min_ps", "top_ks"):
        p = cbk._Sampling(1.0, 1.0, 0.0, 0)
        setattr(p, name, A)
        need = cbk.load_library().cbk_sample_workspace_bytes(ctypes.byref(p), 100, 4)
        assert (need > 0) == (name == "temperatures")


def test_init(cbk):
    lib = cbk.load_library()

    def t(rows, cols, U=300, b=None, words=A):
        return cbk._Tensor(rows, cols, U, cbk.bits_for(U) if b is None else b, A, words)

    def init(gate, up, down, count=2, buffer=A, n=1 << 20):
        arrays = [None if ts is None else (cbk._Tensor * len(ts))(*ts) for ts in (gate, up, down)]
        return lib.cbk_experts_init(*arrays, count, buffer, n, ctypes.byref(cbk._Experts()))
    g, d = [t(64, 32), t(64, 32, 9)], [t(48, 64), t(48, 64)]
    assert lib.cbk_experts_bytes(2) >= 6 * 32 and lib.cbk_experts_bytes(2) % 256 == 0
    assert init(None, g, d) == INVALID and init(g, None, d) == INVALID and init(g, g, None) == INVALID
    assert init(g, g, d, buffer=None) == INVALID and init(g, g, d, count=0) == INVALID and init(g, g, d, count=1025) == INVALID
    assert init(g, [t(64, 32), t(64, 33)], d) == INVALID and init(g, g, [t(48, 64), t(48, 63)]) == INVALID
    assert init([t(64, 32), t(64, 32, b=3)], g, d) == INVALID and init([t(64, 32, words=A + 4)] * 2, g, d) == ALIGN
    assert init(g, g, d, buffer=A + 128) == ALIGN and init(g, g, d, n=100) == CAPACITY
    assert init([t(0, 32)] * 2, [t(0, 32)] * 2, [t(48, 0)] * 2) == INVALID
    assert init([t((1 << 20) + 1, 1)] * 2, [t((1 << 20) + 1, 1)] * 2, [t(1, (1 << 20) + 1)] * 2) == UNSUPPORTED


def test_the_binding_refuses(cbk):
    import torch
    z, x = torch.randn(4, 8), torch.randn(4, 8).bfloat16()
    e, w = torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, 2)
    for call in (lambda: cbk.route(z.half(), 2), lambda: cbk.route(z[0], 2), lambda: cbk.route(z.T, 2), lambda: cbk.route(z, 2, score="tanh"),
                 lambda: cbk.route(z, 2, bias=torch.zeros(7)), lambda: cbk.route(z, 2, bias=torch.zeros(8).double()), lambda: cbk.route(z, -1),
                 lambda: cbk.route(z, 2), lambda: cbk.route(z.expand(4, 8)[:1].expand(4, 8), 2), lambda: cbk.route(z.requires_grad_(), 2),
                 lambda: cbk.route_bwd(z, e.long(), w), lambda: cbk.route_bwd(z, e[:3], w), lambda: cbk.route_bwd(z, e, w.double()),
                 lambda: cbk.route_bwd(z, e, w, out=x), lambda: cbk.sample(z, torch.rand(3)), lambda: cbk.sample(z.half(), torch.rand(4)),
                 lambda: cbk.sample(z, torch.rand(4), temperature=torch.rand(4).double()), lambda: cbk.sample(z, torch.rand(4), top_k=torch.ones(4)),
                 lambda: cbk.sample(z, torch.rand(4)), lambda: cbk.Experts([], [], [])):
        with pytest.raises(ValueError):
            call()
        z = z.detach()
    t = cbk.encode(torch.randn(8, 8).bfloat16()).to("cpu")
    with pytest.raises(ValueError):
        cbk.Experts([t], [t], [t])
    with pytest.raises(ValueError):
        cbk.Experts([t], [t, t], [t])


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_the_headers_are_c99(tmp_path):
    src = tmp_path / "a.c"
    src.write_text('#include "cbk_sample.h"\nint main(void) { return cbk_sample(0, 0, CBK_F32, 0, 0, 0, 0, 0, 0, 0, 0, 0) == CBK_OK; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "a.o")], check=True)
