"""Plain float64 references of the operators in include/cbk_moe.h and include/cbk_sample.h, with bounds on how far fp32
sums and BF16 roundings can take a result from them (the notation is nn_reference's)."""
import math

import torch

import nn_reference as ref
from nn_reference import FUNC, SUM, U16, U32


def route(z, k, score="softmax", bias=None, groups=1, top_groups=None, group_top=1, renormalise=True, scale=1.0):
    """(experts, weights in float64), token by token as the header words it."""
    z = z.double().cpu()
    T, E = z.shape
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double().cpu()
    experts, weights = torch.full((T, k), -1, dtype=torch.int32), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        row = z[t].tolist()
        if any(math.isnan(v) or v == math.inf for v in row):
            experts[t], weights[t] = torch.arange(k, dtype=torch.int32), math.nan
            continue
        top = max(row)
        if score == "softmax":
            ex = [math.exp(v - top) if v > -math.inf else 0.0 for v in row]
            s = [v / max(sum(ex), 1e-300) for v in ex]
        else:
            s = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in row]
        c = [s[e] + float(b[e]) for e in range(E)]
        if any(math.isnan(v) for v in c):
            experts[t], weights[t] = torch.arange(k, dtype=torch.int32), math.nan
            continue
        can = [e for e in range(E) if row[e] > -math.inf and float(b[e]) > -math.inf]
        # without a bias scores are in the order of the logits, also where they are equal in 64 bits
        rank = (lambda e: row[e]) if bias is None and not (groups > 1 and group_top == 2) else (lambda e: c[e])
        if groups > 1:
            size = E // groups
            mark = {}
            for g in range(groups):
                best = sorted((rank(e) for e in can if e // size == g), reverse=True)[:group_top]
                if best:
                    mark[g] = sum(best)
            kept = sorted(mark, key=lambda g: (-mark[g], g))[: groups if top_groups is None else top_groups]
            can = [e for e in can if e // size in kept]
        chosen = sorted(can, key=lambda e: (-rank(e), e))[:k]
        if not chosen:
            continue
        if renormalise:  # relative to the largest of the chosen
            log_s = (lambda v: v) if score == "softmax" else (lambda v: min(v, 0.0) - math.log1p(math.exp(-abs(v))))
            top_s = max(log_s(row[e]) for e in chosen)
            w = [math.exp(log_s(row[e]) - top_s) for e in chosen]
        else:
            w = [s[e] for e in chosen]
        if renormalise and sum(w) > 0:
            w = [v / sum(w) for v in w]
        experts[t, : len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        weights[t, : len(chosen)] = torch.tensor(w, dtype=torch.float64) * float(torch.tensor(scale, dtype=torch.float32))
    return experts, weights


def route_bwd(z, experts, dweights, score="softmax", renormalise=True, scale=1.0):
    """(dlogits, bound) for logits with finite rows or rows of -inf; the gradient by autograd in float64.  The bound is what
    some 8 + E roundings of numbers of the gradient's terms leave: every term of it is a product of scores in [0, 1] and a
    gradient of size `most`."""
    z64, e = z.double().cpu().clone(), experts.cpu().long()
    T, E = z64.shape
    inside = (e >= 0) & (e < E)
    empty = (z64 == -math.inf).all(1)
    z64[empty] = 0.0
    z64.requires_grad_(True)
    s = torch.softmax(z64, 1) if score == "softmax" else torch.sigmoid(z64)
    w = torch.where(inside, s.gather(1, torch.where(inside, e, 0)), 0.0)
    if renormalise:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    g = torch.where(inside & ~empty[:, None], dweights.double().cpu(), 0.0) * scale
    (dz,) = torch.autograd.grad(w, z64, g)
    most = g.abs().sum(1, keepdim=True)
    magnitude = z.double().cpu().masked_fill(z.cpu() == -math.inf, 0.0).abs().amax(1, keepdim=True)
    return dz, (FUNC + (16 + E + 4 * magnitude) * U32) * most + ref.TINY


def _slots(experts, count):
    e = experts.cpu().long()
    return [torch.nonzero(e == i, as_tuple=True) for i in range(count)]


def _hidden(act, x, wg, wu):
    """(g, its bound, u, its bound, act(g), its bound, H, its bound before rounding)"""
    g, eg = ref.product(x, wg)
    u, eu = ref.product(x, wu)
    a, _, b1, _ = ref.act(act, g)
    ea = b1 * eg + FUNC * (a.abs() + g.abs() * 0.3)
    h = a * u
    return g, eg, u, eu, a, ea, h, ea * u.abs() + (a.abs() + ea) * eu + U32 * h.abs()


def experts(act, wg, wu, wd, x, chosen, weights):
    """(Y, bound) for lists of BF16 tensors."""
    T, k = chosen.shape
    y = torch.zeros(T, wd[0].shape[0], dtype=torch.float64)
    e, mag = torch.zeros_like(y), torch.zeros_like(y)
    for i, (t, j) in enumerate(_slots(chosen, len(wg))):
        if t.numel() == 0:
            continue
        h, bh = ref.ffn(act, x[t], wg[i], wu[i])
        d = wd[i].double()
        part = h @ d.T
        off = bh @ d.abs().T + SUM * d.shape[1] * U32 * ((h.abs() + bh) @ d.abs().T)
        w = weights.double().cpu()[t, j][:, None]
        y.index_add_(0, t, w * part)
        e.index_add_(0, t, w.abs() * off)
        mag.index_add_(0, t, (w * part).abs() + w.abs() * off)
    return y, ref.rounded(y, e + (k + 2) * U32 * mag)


def experts_bwd(act, wg, wu, wd, x, chosen, weights, dy):
    """((dX, bound), (dweights, bound))"""
    T, k = chosen.shape
    dx = torch.zeros(T, x.shape[1], dtype=torch.float64)
    ex, mag = torch.zeros_like(dx), torch.zeros_like(dx)
    dw, edw = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for i, (t, j) in enumerate(_slots(chosen, len(wg))):
        if t.numel() == 0:
            continue
        g, eg, u, eu, a, ea, h, eh = _hidden(act, x[t], wg[i], wu[i])
        _, s, _, b2 = ref.act(act, g)
        es = b2 * eg + FUNC * (1 + s.abs() + g.abs() * 0.3)
        D, eD = ref.product(dy[t], wd[i].T)
        dw[t, j] = (h * D).sum(1)
        edw[t, j] = (eh * D.abs() + (h.abs() + eh) * eD).sum(1) + (h.shape[1] + 8) * U32 * (h.abs() * D.abs()).sum(1)
        w = weights.double().cpu()[t, j][:, None]
        dh, edh = w * D, w.abs() * eD + U32 * (w * D).abs()
        dg, du = dh * u * s, dh * a
        top = dh.abs() + edh
        bg = ref.rounded(dg, edh * (u * s).abs() + top * (eu * (s.abs() + es) + u.abs() * es) + 2 * U32 * dg.abs())
        bu = ref.rounded(du, edh * a.abs() + top * ea + U32 * du.abs())
        G, U = wg[i].double(), wu[i].double()
        part = dg @ G + du @ U
        size = (dg.abs() + bg) @ G.abs() + (du.abs() + bu) @ U.abs()
        off = bg @ G.abs() + bu @ U.abs() + SUM * 2 * G.shape[0] * U32 * size
        dx.index_add_(0, t, part)
        ex.index_add_(0, t, off)
        mag.index_add_(0, t, part.abs() + off)
    return (dx, ref.rounded(dx, ex + (k + 10) * U32 * mag)), (dw, edw + ref.TINY)


class Sum:
    """A running sum whose roundings are kept beside it (2 ** -52 of a large first term, added up a million times, would
    be 0.1 % of terms some 10 ** -13 of it)."""

    def __init__(self):
        self.high = self.low = 0.0

    def add(self, v):
        s = self.high + v
        b = s - self.high
        self.low += (self.high - (s - b)) + (v - b)
        self.high = s

    def less(self, limit):
        return (self.high - limit) + self.low


def sample(z, uniform, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of one row, as the header words it, with numbers."""
    z = [float(v) for v in z]
    if any(math.isnan(v) for v in z) or max(z) == -math.inf or math.isnan(temperature):
        return -1, math.nan
    top = max(z)
    order = sorted((i for i in range(len(z)) if z[i] > -math.inf), key=lambda i: (-z[i], i))
    if temperature <= 0:
        return order[0], 0.0

    def x(i):
        if top == math.inf:
            return 0.0 if z[i] == top else -math.inf
        return (z[i] - top) / temperature
    p = {i: math.exp(x(i)) for i in order}
    if top_k > 0:
        order = order[:int(top_k)]
    if min_p > 0:
        border = math.log(min(min_p, 1.0))
        order = [i for i in order if x(i) >= border]
    if top_p < 1:
        want = max(top_p, 0.0) * math.fsum(p[i] for i in order)
        kept, before = [], Sum()
        for i in order:
            if kept and before.less(want) >= 0:
                break
            kept.append(i)
            before.add(p[i])
        order = kept
    total = math.fsum(p[i] for i in order)
    u = uniform if uniform >= 0 else 0.0
    drawn, run = None, Sum()
    for i in sorted(order):
        if p[i] > 0:
            run.add(p[i])
            drawn = i
            if run.less(u * total) > 0:
                break
    return drawn, x(drawn) - math.log(total)
