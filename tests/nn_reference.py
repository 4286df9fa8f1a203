"""Plain float64 references of the operators in include/cbk_nn.h, with bounds on how far fp32 sums
and BF16 roundings can take a result from them.

Notation of the bounds: u32 = 2^-24 and u16 = 2^-8 are half a step of fp32 and of BF16 relative to
the value.  A product of two BF16 numbers is exact in fp32, so a sum of n of them, in any order, is
off by at most n u32 sum |x w| to first order; the matrix instructions are granted twice that
(SUM = 2) for what they round inside.  A function evaluated in fp32 is granted FUNC = 16 u32
relative (the fast exponential's and the division's few units, and the argument's own rounding is
counted separately)."""
import math

import torch

U32 = 2.0 ** -24
U16 = 2.0 ** -8
SUM = 2.0
FUNC = 16 * U32
TINY = 2.0 ** -126  # results below the smallest normal number are off by at most this


def product(x, w):
    """(x . w^T, its fp32 error bound) for BF16-valued x [T][K] and w [N][K]."""
    x, w = x.double(), w.double()
    return x @ w.T, SUM * max(1, x.shape[1]) * U32 * (x.abs() @ w.abs().T)


def rounded(y, err):
    """The bound after rounding y (off by err) to BF16."""
    return err + U16 * (y.abs() + err) + TINY


def act(name, z):
    """(act, act', a bound on |act'|, a bound on |act''|) in float64."""
    z = z.double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s)), 1.1, 0.5
    if name == "gelu":
        p = torch.special.ndtr(z)
        d = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return z * p, p + z * d, 1.13, 0.8
    c = math.sqrt(8 / math.pi)
    s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z), 1.13, 1.0


def linear(x, w):
    y, e = product(x, w)
    return y, rounded(y, e)


def linear_dx(dy, w):
    return linear(dy, w.T)


def ffn(name, x, wg, wu):
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a, _, b1, _ = act(name, g)
    ea = b1 * eg + FUNC * (a.abs() + g.abs() * 0.3)  # z f(z): f in [0, 1] off by FUNC relative, |z| f' bounded
    h = a * u
    return h, rounded(h, ea * u.abs() + (a.abs() + ea) * eu + U32 * h.abs())


def ffn_bwd(name, x, wg, wu, dh):
    """((dX, bound), (dG, bound), (dU, bound))"""
    dh = dh.double()
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a, d, b1, b2 = act(name, g)
    ea = b1 * eg + FUNC * (a.abs() + g.abs() * 0.3)
    ed = b2 * eg + FUNC * (1 + d.abs() + g.abs() * 0.3)
    dg, du = dh * u * d, dh * a
    eg2 = dh.abs() * (eu * (d.abs() + ed) + u.abs() * ed) + 2 * U32 * dg.abs()
    eu2 = dh.abs() * ea + U32 * du.abs()
    bg, bu = rounded(dg, eg2), rounded(du, eu2)
    wg, wu = wg.double(), wu.double()
    dx = dg @ wg + du @ wu
    # the products take dG and dU as rounded (bg, bu); the sum runs over both tensors' rows
    mag = (dg.abs() + bg) @ wg.abs() + (du.abs() + bu) @ wu.abs()
    e = bg @ wg.abs() + bu @ wu.abs() + SUM * 2 * max(1, wg.shape[0]) * U32 * mag
    return (dx, rounded(dx, e)), (dg, bg), (du, bu)


def xent(x, w, labels, ignore):
    """((loss, bound), (lse, bound))"""
    z, ez = product(x, w)
    lse = torch.logsumexp(z, 1)
    keep = labels != ignore
    at = torch.where(keep, labels, 0)
    loss = torch.where(keep, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    # a sum of exponentials, each off by its argument's error and a few units, and its logarithm
    top = z.abs().amax(1) + ez.amax(1)
    el = ez.amax(1) + (SUM * w.shape[0] + 64 + 4 * top) * U32 + 4 * U32 * lse.abs()
    return (loss, torch.where(keep, el + ez.amax(1) + U32 * (lse.abs() + top), 0.0)), (lse, el)


def xent_bwd(x, w, labels, dloss, ignore):
    """(dX, bound), for the lse that the forward call gives."""
    z, ez = product(x, w)
    (_, _), (lse, el) = xent(x, w, labels, ignore)
    keep = labels != ignore
    p = torch.exp(z - lse[:, None])
    ep = p * (ez + el[:, None] + (z - lse[:, None]).abs() * U32 + FUNC)
    p[torch.nonzero(keep)[:, 0], labels[keep]] -= 1
    bp = rounded(p, ep + U32)
    s = torch.where(keep, dloss.double(), 0.0)[:, None]
    wd = w.double()
    dx = p @ wd
    e = bp @ wd.abs() + SUM * w.shape[0] * U32 * ((p.abs() + bp) @ wd.abs())
    dx, e = dx * s, e * s.abs()
    return dx, rounded(dx, e + U32 * dx.abs())


def assert_within(got, want, bound, what):
    got, want, bound = got.double().cpu(), want.cpu(), bound.cpu()
    assert got.shape == want.shape, what
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
                             f"{got[i].item()} for {want[i].item()}, bound {bound[i].item()}")
