"""The workloads of the operators that run a model's training and scoring steps on codebook-compressed weights: products
for any number of tokens and their input gradients, the gated feed-forward block, and the cross entropy over a
compressed output head.  Each case is one call (or, for a training step of the head, the loss and its gradient).

A compressed tensor is what include/cbk.h defines: the ascending distinct 16-bit patterns and b-bit indices, packed
least significant bit first.  The weights are drawn here from the seed and packed with plain tensor operations."""
import math

import torch

own = False

DEVICE = "cuda"
IGNORE = -100


# ---------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step: the gate and up projections of a 7B-shaped block
        {"name": "ffn_t1", "op": "ffn", "tokens": 1, "cols": 4096, "rows": 11008, "act": "silu", "spread": "gauss"},
        # a decode step that serves 13 sequences, 70B-shaped block, heavy-tailed weights
        {"name": "ffn_t13_70b", "op": "ffn", "tokens": 13, "cols": 8192, "rows": 28672, "act": "silu", "spread": "heavy"},
        # a short prompt's prefill
        {"name": "ffn_t200", "op": "ffn", "tokens": 200, "cols": 4096, "rows": 11008, "act": "silu", "spread": "gauss"},
        # a training batch of 2048 tokens
        {"name": "ffn_t2048", "op": "ffn", "tokens": 2048, "cols": 4096, "rows": 11008, "act": "silu", "spread": "gauss"},
        # a small model with odd sizes, one ragged batch
        {"name": "ffn_bwd_t45_odd", "op": "ffn_bwd", "tokens": 45, "cols": 1001, "rows": 2730, "act": "gelu", "spread": "gauss"},
        # the training batch's backward pass
        {"name": "ffn_bwd_t2048", "op": "ffn_bwd", "tokens": 2048, "cols": 4096, "rows": 11008, "act": "silu", "spread": "gauss"},
        # the down projection of a batch of 64 sequences
        {"name": "linear_t64", "op": "linear", "tokens": 64, "cols": 11008, "rows": 4096, "spread": "gauss"},
        # tuning a prompt of a few tokens through an attention projection
        {"name": "linear_dx_t8", "op": "linear_dx", "tokens": 8, "cols": 4096, "rows": 4096, "spread": "gauss"},
        # the down projection's backward pass of the training batch
        {"name": "linear_dx_t2048", "op": "linear_dx", "tokens": 2048, "cols": 11008, "rows": 4096, "spread": "gauss"},
        # scoring a few candidate tokens
        {"name": "xent_t7", "op": "xent", "tokens": 7, "cols": 4096, "rows": 32000, "spread": "gauss"},
        # a training step's loss and gradient over a large vocabulary, a short ragged batch
        {"name": "xent_step_t300_v128k", "op": "xent_step", "tokens": 300, "cols": 4096, "rows": 128000, "spread": "gauss"},
        # a training step's loss and gradient, the whole batch
        {"name": "xent_step_t2048", "op": "xent_step", "tokens": 2048, "cols": 4096, "rows": 32000, "spread": "heavy"},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_bwd", "linear", "linear_dx", "xent", "xent_step"])
    tokens = _log_int(rng, 1, 2048)
    cols = _log_int(rng, 256, 8192)
    rows = _log_int(rng, 8000, 128000) if op.startswith("xent") else _log_int(rng, 256, 28672)
    kind = rng.choice(["even", "even", "units", "odd"])  # most models' widths are multiples of 64 or more
    if kind == "even":
        cols, rows = max(128, cols // 128 * 128), max(128, rows // 128 * 128)
    elif kind == "units":
        cols = max(64, cols // 64 * 64)
    else:
        cols, rows = cols | 1, rows | 1
    # no more than the largest listed cases, in weights and in products
    weights = 2 if op.startswith("ffn") else 1
    rows = min(rows, 400_000_000 // (cols * weights))
    passes = {"ffn": 2, "ffn_bwd": 4, "linear": 1, "linear_dx": 1, "xent": 1, "xent_step": 3}[op]
    tokens = max(1, min(tokens, 750_000_000_000 // (passes * rows * cols)))
    case = {"op": op, "tokens": tokens, "cols": cols, "rows": rows, "spread": rng.choice(["gauss", "heavy", "coarse"])}
    if op.startswith("ffn"):
        case["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
    return case


# --------------------------------------------------------------------------------------------------------- inputs

def _generator(seed, what):
    return torch.Generator(device=DEVICE).manual_seed((seed * 1000003 + what) % (1 << 62))


def _weights(case, seed, what):
    """The weights of one tensor, [rows][cols] bfloat16."""
    g = _generator(seed, what)
    w = torch.randn((case["rows"], case["cols"]), generator=g, device=DEVICE) * 0.02
    if case["spread"] == "heavy":  # a few large weights in every row
        w *= torch.exp(0.5 * torch.randn(w.shape, generator=g, device=DEVICE))
    w = w.bfloat16()
    if case["spread"] == "coarse":  # three mantissa bits, as weights that were once quantised have
        w = (w.view(torch.int16) & ~0xF).view(torch.bfloat16)
    return w


def _pack(w):
    """(codebook int16[U], words int32, U, b) of bfloat16 weights."""
    patterns = w.reshape(-1).view(torch.int16).int() & 0xFFFF
    present = torch.bincount(patterns, minlength=65536) > 0
    codebook = torch.nonzero(present).reshape(-1)
    U = codebook.numel()
    b = (U - 1).bit_length()
    index = (torch.cumsum(present, 0) - 1)[patterns]
    n = index.numel()
    index = torch.nn.functional.pad(index, (0, -n % 32)).reshape(-1, 32)
    words = torch.zeros((index.shape[0], b + 1), dtype=torch.int64, device=w.device)
    for i in range(32):
        at, shift = i * b // 32, i * b % 32
        wide = index[:, i] << shift
        words[:, at] |= wide & 0xFFFFFFFF
        words[:, at + 1] |= wide >> 32
    words = words[:, :b].reshape(-1)
    need = (n * b + 31) // 32
    words = torch.nn.functional.pad(words[:need], (0, -need % 4))
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
    codebook = torch.where(codebook >= 1 << 15, codebook - (1 << 16), codebook).short()
    return codebook, words, U, b


def _activations(case, seed):
    """The bfloat16 inputs, labels and upstream gradients of a case."""
    g = _generator(seed, 3)
    T, K, N = case["tokens"], case["cols"], case["rows"]
    a = {}
    if case["op"] != "linear_dx":
        a["x"] = torch.randn((T, K), generator=g, device=DEVICE).bfloat16()
    if case["op"] in ("ffn_bwd", "linear_dx"):
        a["dy"] = (0.01 * torch.randn((T, N), generator=g, device=DEVICE)).bfloat16()
    if case["op"].startswith("xent"):
        labels = torch.randint(0, N, (T,), generator=g, device=DEVICE)
        skip = torch.rand(T, generator=g, device=DEVICE) < 0.05  # padding and prompt tokens
        skip[0] = False
        a["labels"] = torch.where(skip, IGNORE, labels)
        a["dloss"] = (0.5 + torch.rand(T, generator=g, device=DEVICE)) / T  # a weight for each token
    return a


def prepare(case, seed):
    state = {"case": dict(case), **_activations(case, seed)}
    state["tensors"] = []
    for what in range(2 if case["op"].startswith("ffn") else 1):
        codebook, words, U, b = _pack(_weights(case, seed, what))
        state["tensors"].append({"codebook": codebook, "words": words, "U": U, "b": b})
    return state


# ------------------------------------------------------------------------------------------------------ plain form

def _unpack(case, t):
    """The float32 weights of a compressed tensor."""
    n, b = case["rows"] * case["cols"], t["b"]
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
    return t["codebook"][index].view(torch.bfloat16).float().reshape(case["rows"], case["cols"])


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


def _plain(state):
    case, op = state["case"], state["case"]["op"]
    w = [_unpack(case, t) for t in state["tensors"]]
    if op == "linear":
        return (state["x"].float() @ w[0].T).bfloat16()
    if op == "linear_dx":
        return (state["dy"].float() @ w[0]).bfloat16()
    x = state["x"].float()
    if op.startswith("ffn"):
        gate, up = x @ w[0].T, x @ w[1].T
        a, slope = _act(case["act"], gate)
        if op == "ffn":
            return (a * up).bfloat16()
        dh = state["dy"].float()
        dgate, dup = dh * up * slope, dh * a
        return (dgate @ w[0] + dup @ w[1]).bfloat16(), dgate.bfloat16(), dup.bfloat16()
    logits = x @ w[0].T
    top = logits.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(1))
    labels, counted = state["labels"], state["labels"] != IGNORE
    at = torch.where(counted, labels, 0)[:, None]
    loss = torch.where(counted, lse - logits.gather(1, at)[:, 0], 0.0)
    if op == "xent":
        return loss, lse
    scale = torch.where(counted, state["dloss"], 0.0)[:, None]
    dlogits = torch.exp(logits - lse[:, None]) * scale
    dlogits.scatter_add_(1, at, -scale)
    return loss, lse, (dlogits @ w[0]).bfloat16()


def run(state):
    if not own:
        return _plain(state)
    import fly_decode_amd as cbk

    case, op = state["case"], state["case"]["op"]
    w = [cbk.Compressed(case["rows"], case["cols"], t["U"], t["b"], t["codebook"], t["words"]) for t in state["tensors"]]
    if op == "linear":
        return cbk.linear(w[0], state["x"])
    if op == "linear_dx":
        return cbk.linear_dx(w[0], state["dy"])
    if op == "ffn":
        return cbk.ffn_gated(w[0], w[1], state["x"], act=case["act"])
    if op == "ffn_bwd":
        return cbk.ffn_gated_bwd(w[0], w[1], state["x"], state["dy"], act=case["act"])
    loss, lse = cbk.xent(w[0], state["x"], state["labels"], ignore_index=IGNORE)
    if op == "xent":
        return loss, lse
    return loss, lse, cbk.xent_bwd(w[0], state["x"], state["labels"], lse, state["dloss"], ignore_index=IGNORE)


# ---------------------------------------------------------------------------------------------------- work and truth

def work(case):
    T, K, N, op = case["tokens"], case["cols"], case["rows"], case["op"]
    # the index width that this many weights of this spread take
    b = 9 if case["spread"] == "coarse" else 13 if K * N > (2_000_000 if case["spread"] == "heavy" else 6_000_000) else 12
    weights = K * N * b / 8 * (2 if op.startswith("ffn") else 1)
    product = 2.0 * T * K * N
    if op == "linear":
        return {"bytes": weights + 2 * T * (K + N), "flops": product}
    if op == "linear_dx":
        return {"bytes": weights + 2 * T * (K + N), "flops": product}
    if op == "ffn":
        return {"bytes": weights + 2 * T * (K + N), "flops": 2 * product}
    if op == "ffn_bwd":  # the projections are not kept by the forward pass: their products, and the gradient's two
        return {"bytes": weights + 2 * T * (K + N) + 2 * T * (K + 2 * N), "flops": 4 * product}
    if op == "xent":
        return {"bytes": weights + 2 * T * K + 16 * T, "flops": product}
    # the loss, and the gradient that has the logits to compute again because nothing of their size is kept
    return {"bytes": 2 * weights + 6 * T * K + 40 * T, "flops": 3 * product}


def exact(case, seed):
    """The operators' definitions in float64, on the weights as they were before they were packed."""
    a = {k: v.double() if v.is_floating_point() else v for k, v in _activations(case, seed).items()}
    op = case["op"]
    W = _weights(case, seed, 0).double()
    if op == "linear":
        return torch.matmul(a["x"], W.t())
    if op == "linear_dx":
        return torch.matmul(a["dy"], W)
    if op.startswith("ffn"):
        V = _weights(case, seed, 1).double()
        gate = torch.matmul(a["x"], W.t()).requires_grad_(op == "ffn_bwd")
        up = torch.matmul(a["x"], V.t()).requires_grad_(op == "ffn_bwd")
        if case["act"] == "silu":
            hidden = gate * torch.sigmoid(gate)
        elif case["act"] == "gelu":
            hidden = gate * torch.special.ndtr(gate)
        else:
            hidden = gate * torch.sigmoid(math.sqrt(8 / math.pi) * (gate + 0.044715 * gate ** 3))
        hidden = hidden * up
        if op == "ffn":
            return hidden
        dgate, dup = torch.autograd.grad(hidden, (gate, up), a["dy"])
        return torch.matmul(dgate, W) + torch.matmul(dup, V), dgate, dup
    z = torch.matmul(a["x"], W.t())
    lse = torch.logsumexp(z, 1)
    keep = a["labels"] != IGNORE
    rows = torch.nonzero(keep).reshape(-1)
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, a["labels"][rows]]
    if op == "xent":
        return loss, lse
    d = torch.softmax(z, 1)
    d[rows, a["labels"][rows]] -= 1
    d *= (a["dloss"] * keep)[:, None]
    return loss, lse, torch.matmul(d, W)
