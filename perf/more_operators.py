"""The workloads of the operators that a compressed model with experts needs between its attention and its next token:
routing tokens to experts, the experts' gated feed-forward blocks over codebook-compressed weights, the gradients of
both, and drawing the next token from a head's logits.  Each case is one call.

A compressed tensor is what include/cbk.h defines: the ascending distinct 16-bit patterns and b-bit indices, packed
least significant bit first.  The weights are drawn here from the seed and packed with plain tensor operations."""
import math

import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------------------------------------------------- cases

def listed():
    layer = {"experts": 32, "k": 4, "cols": 4096, "rows": 2048, "act": "silu", "spread": "gauss"}
    return [
        # one token of a decode step
        {"name": "route_t1", "op": "route", "tokens": 1, "experts": 64, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renormalise": True, "scale": 1.0, "dtype": "float32"},
        # a training batch over many experts, balanced by a bias, its experts from half of the groups
        {"name": "route_t4096_groups", "op": "route", "tokens": 4096, "experts": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "renormalise": True, "scale": 2.5, "dtype": "float32"},
        # a small model's ragged batch, an odd number of experts, scores as the linear operator rounds them
        {"name": "route_bwd_t45_odd", "op": "route_bwd", "tokens": 45, "experts": 61, "k": 5, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renormalise": False, "scale": 1.0, "dtype": "bfloat16"},
        # a long training batch's backward pass
        {"name": "route_bwd_t16384", "op": "route_bwd", "tokens": 16384, "experts": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renormalise": True, "scale": 1.0, "dtype": "float32"},
        # one token of a decode step: four of 32 experts are read
        {"name": "experts_t1", "op": "experts", "tokens": 1, **layer},
        # a decode step that serves 48 sequences: every expert is read, for a few tokens each
        {"name": "experts_t48", "op": "experts", "tokens": 48, **layer},
        # a small model with odd sizes, a ragged batch's backward pass
        {"name": "experts_bwd_t45_odd", "op": "experts_bwd", "tokens": 45, "experts": 7, "k": 2, "cols": 1001, "rows": 683,
         "act": "gelu", "spread": "gauss"},
        # a training batch of 2048 tokens
        {"name": "experts_t2048", "op": "experts", "tokens": 2048, **layer},
        # its backward pass
        {"name": "experts_bwd_t2048", "op": "experts_bwd", "tokens": 2048, **layer},
        # the next token of one sequence
        {"name": "sample_t1", "op": "sample", "tokens": 1, "vocabulary": 32000, "filters": "each", "dtype": "float32"},
        # a serving batch over a large vocabulary, each sequence with its own settings
        {"name": "sample_t192_v128k", "op": "sample", "tokens": 192, "vocabulary": 128000, "filters": "each", "dtype": "float32"},
        # a batch drawn by temperature alone, odd vocabulary, logits as the linear operator rounds them
        {"name": "sample_t64_plain", "op": "sample", "tokens": 64, "vocabulary": 50257, "filters": "none", "dtype": "bfloat16"},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "experts", "experts", "experts_bwd", "sample"])
    if op.startswith("route"):
        groups = rng.choice([1, 1, 4, 8])
        n = max(4, _log_int(rng, 4, 512) // groups) * groups
        top = rng.randint(max(1, groups // 4), groups)
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "experts": n, "k": rng.randint(1, min(8, n // groups * top)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups, "top_groups": top,
                "renormalise": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["float32", "bfloat16"])}
    if op == "sample":
        V = _log_int(rng, 500, 200000)
        return {"op": op, "tokens": max(1, min(_log_int(rng, 1, 512), 24_000_000 // V)), "vocabulary": V,
                "filters": rng.choice(["each", "each", "none"]), "dtype": rng.choice(["float32", "bfloat16"])}
    n = _log_int(rng, 4, 64)
    k = rng.randint(1, min(n, 8))
    cols, rows = _log_int(rng, 256, 8192), _log_int(rng, 128, 4096)
    kind = rng.choice(["even", "even", "units", "odd"])  # most models' widths are multiples of 64 or more
    if kind == "even":
        cols, rows = max(128, cols // 128 * 128), max(128, rows // 128 * 128)
    elif kind == "units":
        cols, rows = max(64, cols // 64 * 64), max(64, rows // 64 * 64)
    else:
        cols, rows = cols | 1, rows | 1
    # no more than the largest listed cases, in weights and in products
    n = max(min(n, 268_000_000 // (cols * rows)), k)
    tokens = max(1, min(_log_int(rng, 1, 2048), 68_000_000_000 // (k * rows * cols)))
    return {"op": op, "tokens": tokens, "experts": n, "k": k, "cols": cols, "rows": rows,
            "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh"]), "spread": rng.choice(["gauss", "heavy", "coarse"])}


# --------------------------------------------------------------------------------------------------------- inputs

def _generator(seed, what):
    return torch.Generator(device=DEVICE).manual_seed((seed * 1000003 + what) % (1 << 62))


def _weights(case, seed, kind):
    """The weights of every expert's tensor of a kind: [experts][rows][cols] bfloat16, the down projection (2) [experts][cols][rows]."""
    shape = (case["cols"], case["rows"]) if kind == 2 else (case["rows"], case["cols"])
    g = _generator(seed, 10 + kind)
    w = torch.randn((case["experts"], *shape), generator=g, device=DEVICE)
    if case["spread"] == "heavy":  # a few large weights in every row
        w *= torch.exp(0.5 * torch.randn(w.shape, generator=g, device=DEVICE))
    w = w.mul_(0.02).bfloat16()
    if case["spread"] == "coarse":  # three mantissa bits, as weights that were once quantised have
        w = (w.view(torch.int16) & ~0xF).view(torch.bfloat16)
    return w


def _pack_alike(index, b):
    """b-bit indices [tensors][n], packed: int32 [tensors][words], whole groups of four words."""
    n = index.shape[1]
    index = torch.nn.functional.pad(index, (0, -n % 32)).reshape(index.shape[0], -1, 32)
    words = torch.zeros((*index.shape[:2], b + 1), dtype=torch.int64, device=index.device)
    for i in range(32):
        at, shift = i * b // 32, i * b % 32
        wide = index[:, :, i].long() << shift
        words[:, :, at] |= wide & 0xFFFFFFFF
        words[:, :, at + 1] |= wide >> 32
    words = words[:, :, :b].reshape(index.shape[0], -1)
    need = (n * b + 31) // 32
    words = torch.nn.functional.pad(words[:, :need], (0, -need % 4))
    return torch.where(words >= 1 << 31, words - (1 << 32), words).int()


def _pack(w):
    """The compressed tensors of w [tensors][rows][cols]: (codebook int16[U], words int32, U, b) each."""
    count, n = w.shape[0], w.shape[1] * w.shape[2]
    patterns = w.reshape(count, n).view(torch.int16).int() & 0xFFFF
    present = torch.zeros((count, 65536), dtype=torch.bool, device=w.device)
    for e in range(count):
        present[e, patterns[e].long()] = True
    place = torch.cumsum(present, 1, dtype=torch.int32) - 1
    index = torch.stack([place[e][patterns[e].long()] for e in range(count)])
    sizes = present.sum(1).tolist()
    tensors = [None] * count
    for b in sorted({(U - 1).bit_length() for U in sizes}):
        alike = [e for e in range(count) if (sizes[e] - 1).bit_length() == b]
        words = _pack_alike(index[alike], b)
        for i, e in enumerate(alike):
            codebook = torch.nonzero(present[e]).reshape(-1)
            codebook = torch.where(codebook >= 1 << 15, codebook - (1 << 16), codebook).short()
            tensors[e] = {"codebook": codebook, "words": words[i].clone(), "U": sizes[e], "b": b}
    return tensors


def _inputs(case, seed):
    """What a case takes beside its weights."""
    g = _generator(seed, 3)
    T, op = case["tokens"], case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEVICE)

    a = {}
    if op == "sample":
        V = case["vocabulary"]
        z = 2.5 * normal(T, V)
        z[uniform(T, V) < 0.01] = -math.inf  # tokens that may not come next
        a["logits"] = z.to(getattr(torch, case["dtype"]))
        a["uniform"] = uniform(T)
        a["temperature"] = 0.6 + 0.7 * uniform(T)
        if case["filters"] == "each":  # a sequence's own settings, a few without one filter or another, a few greedy
            a["temperature"] = torch.where(uniform(T) < 0.05, 0.0, a["temperature"])
            a["top_k"] = torch.tensor([0, 20, 50, 200, 1000], device=DEVICE)[(5 * uniform(T)).long()].int()
            a["top_p"] = torch.tensor([1.0, 0.95, 0.9, 0.6], device=DEVICE)[(4 * uniform(T)).long()]
            a["min_p"] = torch.tensor([0.0, 0.0, 0.02, 0.1], device=DEVICE)[(4 * uniform(T)).long()]
        return a
    n, k = case["experts"], case["k"]
    if op.startswith("route"):
        z = 1.5 * normal(T, n) + 0.5 * normal(1, n)  # experts differ in how much they are liked
        z[(uniform(T) < 0.02) & (torch.arange(T, device=DEVICE) > 0)] = -math.inf  # padding
        a["logits"] = z.to(getattr(torch, case["dtype"]))
        a["bias"] = 0.05 * normal(n) if case["bias"] else None
        if op == "route_bwd":
            a["chosen"] = _route(case, a["logits"], a["bias"])[0]
            a["dweights"] = normal(T, k)
        return a
    z = normal(T, n) + 0.5 * normal(1, n)
    weights, chosen = torch.topk(torch.softmax(z, 1), k, dim=1)
    padding = (uniform(T) < 0.02) & (torch.arange(T, device=DEVICE) > 0)
    a["chosen"] = torch.where(padding[:, None], -1, chosen).int()
    a["weights"] = torch.where(padding[:, None], 0.0, weights / weights.sum(1, keepdim=True))
    a["x"] = normal(T, case["cols"]).bfloat16()
    if op == "experts_bwd":
        a["dy"] = (0.01 * normal(T, case["cols"])).bfloat16()
    return a


def prepare(case, seed):
    state = {"case": dict(case), **_inputs(case, seed)}
    if case["op"].startswith("experts"):
        state["tensors"] = [_pack(_weights(case, seed, kind)) for kind in range(3)]
    return state


# ------------------------------------------------------------------------------------------------------ plain form

def _route(case, logits, bias):
    """(experts int32 [T][k], weights float32 [T][k]).  In 64 bits, since two scores may be next to each other."""
    z = logits.double()
    T, n = z.shape
    k, groups = case["k"], case["groups"]
    if case["score"] == "softmax":
        top = z.amax(1, keepdim=True)
        e = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        s = 1 / (1 + torch.exp(-z))
    c = s if bias is None else s + bias.double()
    c = torch.where(z == -math.inf, -math.inf, c)  # never chosen
    if groups > 1:
        mark = torch.sort(c.view(T, groups, -1), dim=2, descending=True)[0][:, :, : 1 if bias is None else 2].sum(2)
        order = torch.sort(mark, dim=1, descending=True, stable=True)[1]
        kept = torch.zeros_like(mark, dtype=torch.bool).scatter_(1, order[:, : case["top_groups"]], True)
        c = torch.where(kept[:, :, None], c.view(T, groups, -1), -math.inf).view(T, n)
    c, chosen = torch.sort(c, dim=1, descending=True, stable=True)
    c, chosen = c[:, :k], chosen[:, :k]
    w = torch.where(c == -math.inf, 0.0, s.gather(1, chosen))
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return torch.where(c == -math.inf, -1, chosen).int(), (w * case["scale"]).float()


def _route_bwd(case, logits, chosen, dweights):
    z, d = logits.float(), dweights * case["scale"]
    there = chosen >= 0
    at = torch.where(there, chosen, 0).long()
    d = torch.where(there, d, 0.0)
    if case["score"] == "softmax":
        top = z.amax(1, keepdim=True)
        e = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-30)
    else:
        s = 1 / (1 + torch.exp(-z))
    w = torch.where(there, s.gather(1, at), 0.0)
    if case["renormalise"]:
        total = w.sum(1, keepdim=True).clamp_min(1e-30)
        d = (d - (d * w).sum(1, keepdim=True) / total) / total
        d = torch.where(there, d, 0.0)
    ds = torch.zeros_like(z).scatter_add_(1, at, d)
    if case["score"] == "softmax":
        dz = s * (ds - (d * w).sum(1, keepdim=True))
    else:
        dz = ds * s * (1 - s)
    return dz.to(logits.dtype)


def _unpack(rows, cols, t):
    """The float32 weights of a compressed tensor."""
    n, b = rows * cols, t["b"]
    if b == 0:
        index = torch.zeros(n, dtype=torch.int64, device=DEVICE)
    else:
        words = t["words"].long() & 0xFFFFFFFF
        groups = (n + 31) // 32
        words = torch.nn.functional.pad(words, (0, max(0, groups * b - words.numel())))[: groups * b].reshape(groups, b)
        words = torch.nn.functional.pad(words, (0, 1))
        bit = torch.arange(32, device=DEVICE) * b
        low = words[:, bit // 32] >> (bit % 32)
        high = words[:, bit // 32 + 1] << (32 - bit % 32)
        index = ((low | high) & ((1 << b) - 1)).reshape(-1)[:n]
    return t["codebook"][index].view(torch.bfloat16).float().reshape(rows, cols)


def _act(name, z):
    """(act(z), act'(z))"""
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        phi = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _experts(state):
    case, backward = state["case"], state["case"]["op"] == "experts_bwd"
    K, N = case["cols"], case["rows"]
    chosen, weights, x = state["chosen"].long(), state["weights"], state["x"].float()
    out = torch.zeros_like(x)
    dweights = torch.zeros_like(weights)
    for e in torch.unique(chosen).tolist():
        if e < 0:
            continue
        token, slot = torch.nonzero(chosen == e, as_tuple=True)
        gate, up, down = (_unpack(*((K, N) if kind == 2 else (N, K)), state["tensors"][kind][e]) for kind in range(3))
        g, u = x[token] @ gate.T, x[token] @ up.T
        a, slope = _act(case["act"], g)
        w = weights[token, slot][:, None]
        if not backward:
            out.index_add_(0, token, w * ((a * u) @ down.T))
            continue
        d = state["dy"][token].float() @ down
        dweights[token, slot] = (d * a * u).sum(1)
        dh = w * d
        out.index_add_(0, token, (dh * u * slope) @ gate + (dh * a) @ up)
    return (out.bfloat16(), dweights) if backward else out.bfloat16()


def _sample(state):
    z = state["logits"].double()  # in 64 bits: a uniform number may fall next to the border of two tokens
    T, V = z.shape
    each = state["case"]["filters"] == "each"
    greedy = (state["temperature"] == 0)[:, None]
    top = z.amax(1, keepdim=True)
    mass = torch.exp((z - top) / torch.where(greedy, 1.0, state["temperature"][:, None].double()))
    order = torch.sort(z, dim=1, descending=True, stable=True)[1]
    kept = mass.gather(1, order)
    rank = torch.arange(V, device=z.device)[None]
    kept = torch.where(greedy & (rank > 0), 0.0, kept)
    if each:
        k = state["top_k"][:, None]
        kept = torch.where((k > 0) & (rank >= k), 0.0, kept)
        kept = torch.where(kept < state["min_p"][:, None].double(), 0.0, kept)
        before = torch.cumsum(kept, 1) - kept
        kept = torch.where(before >= state["top_p"][:, None].double() * kept.sum(1, keepdim=True), 0.0, kept)
    mass = torch.zeros_like(mass).scatter_(1, order, kept)
    sums = torch.cumsum(mass, 1)
    total = sums[:, -1:]
    token = (sums <= state["uniform"][:, None].double() * total).sum(1)
    chance = mass.gather(1, token[:, None]) / total
    return token, torch.log(chance)[:, 0].float()


def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        if op == "route":
            return _route(case, state["logits"], state["bias"])
        if op == "route_bwd":
            return _route_bwd(case, state["logits"], state["chosen"], state["dweights"])
        return _sample(state) if op == "sample" else _experts(state)
    import fly_decode_amd as cbk

    if op == "route":
        return cbk.route(state["logits"], case["k"], score=case["score"], bias=state["bias"], groups=case["groups"],
                         top_groups=case["top_groups"], group_top=1 if state["bias"] is None else 2,
                         renormalise=case["renormalise"], scale=case["scale"])
    if op == "route_bwd":
        return cbk.route_bwd(state["logits"], state["chosen"], state["dweights"], score=case["score"],
                             renormalise=case["renormalise"], scale=case["scale"])
    if op == "sample":
        filters = {name: state[name] for name in ("top_k", "top_p", "min_p") if name in state}
        return cbk.sample(state["logits"], state["uniform"], temperature=state["temperature"], **filters)
    if "plan" not in state:  # a program makes it once for a layer
        K, N = case["cols"], case["rows"]
        shapes = [(N, K), (N, K), (K, N)]
        state["plan"] = cbk.Experts(*([cbk.Compressed(*shapes[kind], t["U"], t["b"], t["codebook"], t["words"])
                                       for t in state["tensors"][kind]] for kind in range(3)))
    if op == "experts":
        return cbk.ffn_experts(state["plan"], state["x"], state["chosen"], state["weights"], act=case["act"])
    return cbk.ffn_experts_bwd(state["plan"], state["x"], state["chosen"], state["weights"], state["dy"], act=case["act"])


# ---------------------------------------------------------------------------------------------------- work and truth

def work(case):
    T, op = case["tokens"], case["op"]
    if op == "sample":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": T * case["vocabulary"] * size + T * 32, "flops": 20.0 * T * case["vocabulary"]}
    n, k = case["experts"], case["k"]
    if op.startswith("route"):
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": T * (n * size * (1 if op == "route" else 2) + 8 * k), "flops": 20.0 * T * n}
    K, N = case["cols"], case["rows"]
    # the index width that this many weights of this spread take, and the experts that the tokens' choices leave unread
    b = 9 if case["spread"] == "coarse" else 13 if K * N > (2_000_000 if case["spread"] == "heavy" else 6_000_000) else 12
    read = n * (1 - (1 - k / n) ** T)
    weights = read * 3 * K * N * b / 8
    product = 2.0 * T * k * K * N
    if op == "experts":
        return {"bytes": weights + T * (4 * K + 8 * k), "flops": 3 * product}
    # the projections are not kept by the forward pass: their products, the down projection's gradient, and the two of dX
    return {"bytes": weights + T * (6 * K + 12 * k), "flops": 5 * product}


def exact(case, seed):
    """The operators' definitions in float64, on the weights as they were before they were packed."""
    a = {name: v.double() if v is not None and v.is_floating_point() else v for name, v in _inputs(case, seed).items()}
    T, op = case["tokens"], case["op"]
    if op == "sample":
        return _exact_sample(a)
    if op == "route":
        return _exact_route(case, a)
    if op == "route_bwd":
        z = a["logits"].clone()
        empty = (z == -math.inf).all(1)
        z[empty] = 0.0
        z.requires_grad_(True)
        s = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
        w = s.gather(1, a["chosen"].clamp_min(0).long())
        if case["renormalise"]:
            w = w / w.sum(1, keepdim=True)
        (dz,) = torch.autograd.grad(w * case["scale"], z, torch.where(empty[:, None], 0.0, a["dweights"]))
        return dz
    if 6.0 * T * case["k"] * case["cols"] * case["rows"] > 4.5e11:
        return None
    W = [_weights(case, seed, kind) for kind in range(3)]
    flat = a["chosen"].reshape(-1)
    order = torch.argsort(flat, stable=True)
    ends = torch.searchsorted(flat[order].contiguous(), torch.arange(-1, case["experts"], device=DEVICE), right=True).tolist()
    y = torch.zeros_like(a["x"])
    dw = torch.zeros(flat.shape, dtype=torch.float64, device=DEVICE)
    for e in range(case["experts"]):
        slots = order[ends[e]: ends[e + 1]]
        if slots.numel() == 0:
            continue
        rows = slots // case["k"]
        gate, up, down = (w[e].double() for w in W)
        x = a["x"][rows].requires_grad_(op == "experts_bwd")
        w = a["weights"].reshape(-1)[slots].requires_grad_(op == "experts_bwd")
        p, q = torch.matmul(x, gate.t()), torch.matmul(x, up.t())
        if case["act"] == "silu":
            h = p * torch.sigmoid(p) * q
        elif case["act"] == "gelu":
            h = p * torch.special.ndtr(p) * q
        else:
            h = p * torch.sigmoid(math.sqrt(8 / math.pi) * (p + 0.044715 * p ** 3)) * q
        part = torch.matmul(h, down.t()) * w[:, None]
        if op == "experts_bwd":
            part, dw[slots] = torch.autograd.grad(part, (x, w), a["dy"][rows])
        y.index_put_((rows,), part.detach(), accumulate=True)
    return (y, dw.view(T, -1)) if op == "experts_bwd" else y


def _exact_route(case, a):
    z, T, n, k = a["logits"], case["tokens"], case["experts"], case["k"]
    empty = (z == -math.inf).all(1)
    z = torch.where(empty[:, None], 0.0, z)
    s = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
    c = s + a["bias"] if case["bias"] else s

    def places(v):  # of each value among its row's: how many are larger, or as large and before it
        i = torch.arange(v.shape[1], device=DEVICE)
        first = i[None, :] < i[:, None]
        return torch.cat([((r[:, None, :] > r[:, :, None]) | ((r[:, None, :] == r[:, :, None]) & first)).sum(2) for r in v.split(256)])

    if case["groups"] > 1:
        best = torch.topk(c.view(T, case["groups"], -1), 2 if case["bias"] else 1, dim=2)[0].sum(2)
        kept = places(best) < case["top_groups"]
        c = torch.where(kept.repeat_interleave(n // case["groups"], 1), c, -10.0 ** 9)
    place = places(c)
    chosen = torch.empty((T, n), dtype=torch.int64, device=DEVICE).scatter_(1, place, torch.arange(n, device=DEVICE).expand(T, n))[:, :k]
    w = s.gather(1, chosen)
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return torch.where(empty[:, None], -1, chosen).int(), torch.where(empty[:, None], 0.0, w * case["scale"])


def _exact_sample(a):
    """Row by row, the filters as they are named: what is not among the largest k, what is less likely than min_p times the
    likeliest, then what the likeliest that make up top_p of the rest can do without."""
    tokens, logs = [], []
    for t in range(a["logits"].shape[0]):
        z = a["logits"][t]
        heat = float(a["temperature"][t])
        if heat == 0:
            tokens.append(int(torch.nonzero(z == z.max())[0]))
            logs.append(0.0)
            continue
        p = torch.softmax(z / heat, 0)
        if "top_k" in a:
            k = int(a["top_k"][t])
            if 0 < k < z.numel():
                least = torch.topk(z, k)[0][-1]
                ties = torch.nonzero(z == least).reshape(-1)
                drop = z < least
                drop[ties[k - int((z > least).sum()):]] = True
                p = torch.where(drop, 0.0, p)
            p = torch.where(p < float(a["min_p"][t]) * p.max(), 0.0, p)
            p = p / p.sum()
            order = torch.argsort(p, descending=True, stable=True)
            need = int((torch.cumsum(p[order], 0) < float(a["top_p"][t])).sum()) + 1
            keep = torch.zeros_like(p)
            keep[order[:need]] = p[order[:need]]
            p = keep / keep.sum()
        sums = torch.cumsum(p, 0)
        i = int(torch.searchsorted(sums, a["uniform"][t] * sums[-1], right=True))
        tokens.append(i)
        logs.append(float(torch.log(p[i])))
    return torch.tensor(tokens, device=DEVICE), torch.tensor(logs, dtype=torch.float64, device=DEVICE)
