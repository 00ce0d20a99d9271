"""More operators of a training step and of serving, as measured cases: the gated feed-forward product (two projections, an
activation and their product) with its backward pass, the cross entropy of a projection onto a large vocabulary with its
gradient, and the norm of many gradients with clipping.

``run`` computes them in plain torch where ``own`` is false (32-bit sums, rounded once at the end) and through the library's entry
points where it is true.  ``exact`` gives the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
IGNORE = -100
#: the coefficient of clipping is max_norm / (norm + CLIP_EPS), 1 at most
CLIP_EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
# Gated product, over `tokens` rows of `hidden` values and two weights of `inner` x `hidden`: Y = act(X Wg^T) * (X Wu^T).
#   "gated"           the product alone, as in serving
#   "gated_train"     the product, keeping both projections, then the gradients of X, Wg and Wu from them
#   "gated_backward"  the gradients alone, from X and the weights, where nothing was kept to save memory
# Cross entropy over `vocab` classes of logits X W^T:
#   "loss"            the loss and the log of the sum of exponentials for each token (0 for ignored ones), as in evaluation
#   "loss_train"      the same, then the gradients of X and W for the mean loss over the tokens that count
# Clipping:
#   "clip"            the norm of all gradients and the gradients scaled by it into buffers of their own

def listed():
    return [
        # one token through a feed-forward layer while serving: the weights' bytes
        {"name": "gated one token", "op": "gated", "tokens": 1, "hidden": 4096, "inner": 11008, "dtype": "bf16", "act": "silu"},
        # a batch of tokens being decoded
        {"name": "gated 17 tokens", "op": "gated", "tokens": 17, "hidden": 2048, "inner": 5632, "dtype": "fp16", "act": "gelu_tanh"},
        # a ragged prompt: odd sizes on every side, lines that are no multiple of 16 bytes
        {"name": "gated odd prompt", "op": "gated", "tokens": 1531, "hidden": 1001, "inner": 2741, "dtype": "bf16", "act": "silu"},
        # a training step of a large layer
        {"name": "gated training", "op": "gated_train", "tokens": 8192, "hidden": 4096, "inner": 11008, "dtype": "bf16", "act": "silu"},
        # the backward pass of a layer whose projections were not kept
        {"name": "gated backward", "op": "gated_backward", "tokens": 2048, "hidden": 2048, "inner": 5504, "dtype": "fp16", "act": "gelu_tanh"},
        # the log-probability of one token under a large vocabulary: the weights' bytes
        {"name": "loss one token", "op": "loss", "tokens": 1, "hidden": 4096, "vocab": 32768, "dtype": "bf16", "ignored": 0.0},
        # evaluation of a short text, odd vocabulary
        {"name": "loss evaluation", "op": "loss", "tokens": 512, "hidden": 2048, "vocab": 50257, "dtype": "fp16", "ignored": 0.0},
        # a training step, some tokens padded away
        {"name": "loss training", "op": "loss_train", "tokens": 4096, "hidden": 2048, "vocab": 32768, "dtype": "bf16", "ignored": 0.05},
        # odd sizes on every side, lines that are no multiple of 16 bytes, more padding than tokens
        {"name": "loss training odd", "op": "loss_train", "tokens": 1023, "hidden": 1001, "vocab": 5003, "dtype": "fp16", "ignored": 0.6},
        # a training step over a vocabulary of a hundred thousand, the largest one
        {"name": "loss training large", "op": "loss_train", "tokens": 8192, "hidden": 4096, "vocab": 100003, "dtype": "bf16", "ignored": 0.05},
        # the few small gradients of an adapter: latency
        {"name": "clip small", "op": "clip", "layers": 2, "hidden": 128, "inner": 64, "dtype": "fp32", "out": "fp32"},
        # the gradients of a whole model in 16 bits, scaled into those that its optimiser reads
        {"name": "clip large", "op": "clip", "layers": 20, "hidden": 2048, "inner": 5504, "dtype": "bf16", "out": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _pick(rng, low, high):
    """As _spread; one time in two a multiple of 64 where the range has one."""
    v = _spread(rng, low, high)
    if rng.random() < 0.5 and high >= 64:
        v = min(high // 64 * 64, max(-(-low // 64) * 64, v // 64 * 64))
    return v


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_train", "gated_backward", "loss", "loss_train", "loss_train", "clip"])
    if op == "clip":
        hidden = _pick(rng, 64, 4096)
        inner = _pick(rng, 64, 8192)
        most = max(1, int(1.0e9 / (hidden * (4 * hidden + 3 * inner))))
        return {"op": op, "layers": _spread(rng, 1, min(64, most)), "hidden": hidden, "inner": inner,
                "dtype": rng.choice(["fp32", "bf16", "bf16", "fp16"]), "out": rng.choice(["fp32", "same"])}
    hidden = _pick(rng, 64, 4096)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op.startswith("gated"):
        inner = _pick(rng, 64, 11008)
        return {"op": op, "tokens": _spread(rng, 1, 8192), "hidden": hidden, "inner": inner, "dtype": dtype,
                "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh"])}
    return {"op": op, "tokens": _spread(rng, 1, 8192), "hidden": hidden, "vocab": _pick(rng, 1000, 100003), "dtype": dtype,
            "ignored": rng.choice([0.0, 0.05, 0.5])}


def _shapes(c):
    """The gradients of a decoder's layers: attention and feed-forward matrices, and two vectors of norms a layer."""
    h, i = c["hidden"], c["inner"]
    return [s for _ in range(c["layers"]) for s in ((h, h), (h, h), (h, h), (h, h), (i, h), (i, h), (h, i), (h,), (h,))]


def work(case):
    c = case
    if c["op"] == "clip":
        n = sum(math.prod(s) for s in _shapes(c))
        return {"bytes": n * (SIZE[c["dtype"]] + SIZE[c["dtype"] if c["out"] == "same" else c["out"]]), "flops": 0}
    es, t, h = SIZE[c["dtype"]], c["tokens"], c["hidden"]
    if c["op"].startswith("gated"):
        i = c["inner"]
        x, w, y = t * h * es, 2 * i * h * es, t * i * es
        forward, gradients = 4 * t * i * h, 8 * t * i * h
        if c["op"] == "gated":
            return {"bytes": x + w + y, "flops": forward}
        # (training: Y out, dY in; X and the weights in, their gradients out)
        return {"bytes": 2 * x + 2 * w + (2 if c["op"] == "gated_train" else 1) * y, "flops": forward + gradients}
    v = c["vocab"]
    x, w = t * h * es, v * h * es
    if c["op"] == "loss":
        return {"bytes": x + w + 16 * t, "flops": 2 * t * v * h}
    return {"bytes": 2 * x + 2 * w + 20 * t, "flops": 6 * t * v * h}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _hidden_states(t, h, g, dev):
    """Normalised hidden states: normal values with a few channels that are larger than the others."""
    channel = torch.where(torch.rand(h, generator=g, device=dev) < 0.01, 4.0, 1.0)
    return torch.randn((t, h), generator=g, device=dev) * channel


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = TYPES[c["dtype"]]
    if c["op"] == "clip":
        # views of one buffer, as a bucket of gradients is; sizes differ from tensor to tensor, as layers' gradients do
        shapes = _shapes(c)
        out = TYPES[c["dtype"] if c["out"] == "same" else c["out"]]
        sizes = [math.prod(s) for s in shapes]
        starts, end = [], 0
        for n in sizes:
            starts.append(end)
            end += -(-n // 64) * 64
        flat, into = torch.zeros(end, dtype=dt, device=dev), torch.zeros(end, dtype=out, device=dev)
        grads = [flat[a:a + n].view(s) for a, n, s in zip(starts, sizes, shapes)]
        outs = [into[a:a + n].view(s) for a, n, s in zip(starts, sizes, shapes)]
        for k, t in enumerate(grads):
            t.copy_((1e-3 * (1 + k % 5)) * torch.randn(t.shape, generator=g, device=dev))
        return {"case": c, "grads": grads, "outs": outs, "into": into, "max_norm": 1.0}
    t, h = c["tokens"], c["hidden"]
    x = _hidden_states(t, h, g, dev).to(dt)
    if c["op"].startswith("gated"):
        i = c["inner"]
        wg = (torch.randn((i, h), generator=g, device=dev) / math.sqrt(h)).to(dt)
        wu = (torch.randn((i, h), generator=g, device=dev) / math.sqrt(h)).to(dt)
        s = {"case": c, "x": x, "wg": wg, "wu": wu}
        if c["op"] != "gated":
            # gradients whose size differs from token to token (under fp16's usual loss scaling)
            s["dy"] = (0.1 * torch.randn((t, i), generator=g, device=dev) * torch.exp(torch.randn((t, 1), generator=g, device=dev))).to(dt)
        return s
    v = c["vocab"]
    w = (2 * torch.randn((v, h), generator=g, device=dev) / math.sqrt(h)).to(dt)
    # frequent and rare classes, as words are
    target = (torch.exp(torch.rand(t, generator=g, device=dev, dtype=torch.float64) * math.log(v)).long() - 1).clamp(0, v - 1)
    dropped = torch.rand(t, generator=g, device=dev) < c["ignored"]
    target = torch.where(dropped, IGNORE, target)
    s = {"case": c, "x": x, "w": w, "target": target}
    if c["op"] == "loss_train":
        # the gradient of the mean (under a loss scale in fp16, as is usual there)
        count = (target != IGNORE).sum().clamp(min=1)
        s["dloss"] = ((256.0 if c["dtype"] == "fp16" else 1.0) / count.float()).expand(t)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

GELU_C = math.sqrt(2 / math.pi)


def _act(g, act):
    """(act(g), act'(g)) in g's own type."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    u = GELU_C * (g + 0.044715 * g ** 3)
    th = 1 - 2 / (1 + torch.exp(2 * u))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * GELU_C * (1 + 3 * 0.044715 * g * g)


def _plain_gated(state):
    c = state["case"]
    x, wg, wu = state["x"].float(), state["wg"].float(), state["wu"].float()
    dt = state["x"].dtype
    g, u = x @ wg.t(), x @ wu.t()
    a, d = _act(g, c["act"])
    if c["op"] == "gated":
        return (a * u).to(dt)
    dy = state["dy"].float()
    dg, du = dy * u * d, dy * a
    r = {"dx": (dg @ wg + du @ wu).to(dt), "dwg": (dg.t() @ x).to(dt), "dwu": (du.t() @ x).to(dt)}
    if c["op"] == "gated_train":
        r["y"] = (a * u).to(dt)
    return r


def _plain_loss(state):
    c = state["case"]
    x, w, target = state["x"].float(), state["w"].float(), state["target"]
    dt = state["x"].dtype
    logits = x @ w.t()
    top = logits.amax(dim=1, keepdim=True)
    lse = (logits - top).exp().sum(dim=1).log() + top[:, 0]
    counts = target != IGNORE
    at = torch.where(counts, target, 0)[:, None]
    loss = torch.where(counts, lse - logits.gather(1, at)[:, 0], 0.0)
    if c["op"] == "loss":
        return {"loss": loss, "lse": torch.where(counts, lse, 0.0)}
    p = logits.sub_(lse[:, None]).exp_()
    p.scatter_add_(1, at, torch.full_like(p[:, :1], -1.0))
    p *= torch.where(counts, state["dloss"], 0.0)[:, None]
    return {"loss": loss, "lse": torch.where(counts, lse, 0.0), "dx": (p @ w).to(dt), "dw": (p.t() @ x).to(dt)}


def _plain_clip(state):
    grads = state["grads"]
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads])
    norm = squares.sum().sqrt().float()
    f = (state["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    for g, o in zip(grads, state["outs"]):
        o.copy_(g.float() * f)
    return {"norm": norm, "grads": state["into"]}


def _plain(state):
    op = state["case"]["op"]
    return _plain_clip(state) if op == "clip" else _plain_gated(state) if op.startswith("gated") else _plain_loss(state)


def _own(state):
    import mixed_precision_matmul_gb300 as mpg
    c = state["case"]
    if c["op"] == "clip":
        norm = mpg.clip_grad_norm(state["grads"], state["max_norm"], out=state["outs"])
        return {"norm": norm, "grads": state["into"]}
    if c["op"] == "gated":
        return mpg.gated_gemm(state["x"], state["wg"], state["wu"], act=c["act"])
    if c["op"] == "gated_backward":
        dx, dwg, dwu = mpg.gated_gemm_backward(state["dy"], state["x"], state["wg"], state["wu"], act=c["act"])
        return {"dx": dx, "dwg": dwg, "dwu": dwu}
    if c["op"] == "gated_train":
        y, g, u = mpg.gated_gemm(state["x"], state["wg"], state["wu"], act=c["act"], keep=True)
        dx, dwg, dwu = mpg.gated_gemm_backward(state["dy"], state["x"], state["wg"], state["wu"], act=c["act"], kept=(g, u))
        return {"dx": dx, "dwg": dwg, "dwu": dwu, "y": y}
    loss, lse = mpg.linear_cross_entropy(state["x"], state["w"], state["target"], ignore_index=IGNORE)
    if c["op"] == "loss":
        return {"loss": loss, "lse": lse}
    dx, dw = mpg.linear_cross_entropy_backward(state["x"], state["w"], state["target"], lse, state["dloss"], ignore_index=IGNORE)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _exact_act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * torch.special.erfc(-g / math.sqrt(2.0))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def exact(case, seed):
    c = case
    if work(case)["flops"] > 5e12:       # over about 10 seconds in 64 bits
        return None
    state = prepare(case, seed)
    if c["op"] == "clip":
        if sum(g.numel() for g in state["grads"]) > 4e9:
            return None
        flat = torch.cat([g.reshape(-1) for g in state["grads"]]).double()
        norm = torch.linalg.vector_norm(flat)
        f = torch.clamp(state["max_norm"] / (norm + CLIP_EPS), max=1.0)
        into = torch.zeros(state["into"].shape, dtype=torch.float64, device=flat.device)
        for g, o in zip(state["grads"], state["outs"]):
            a = (o.data_ptr() - state["into"].data_ptr()) // o.element_size()
            into[a:a + g.numel()] = g.reshape(-1).double() * f
        return {"norm": norm, "grads": into}
    x = state["x"].double()
    if c["op"].startswith("gated"):
        wg, wu = state["wg"].double(), state["wu"].double()
        gate = torch.einsum("th,ih->ti", x, wg)
        up = torch.einsum("th,ih->ti", x, wu)
        if c["op"] == "gated":
            return _exact_act(gate, c["act"]) * up
        gate.requires_grad_(True)
        a = _exact_act(gate, c["act"])
        dy = state["dy"].double()
        dgate, = torch.autograd.grad(a, gate, dy * up)
        a = a.detach()
        dup = dy * a
        r = {"dx": torch.einsum("ti,ih->th", dgate, wg) + torch.einsum("ti,ih->th", dup, wu),
             "dwg": torch.einsum("ti,th->ih", dgate, x), "dwu": torch.einsum("ti,th->ih", dup, x)}
        if c["op"] == "gated_train":
            r["y"] = a * up
        return r
    w, target = state["w"].double(), state["target"]
    logits = torch.einsum("th,vh->tv", x, w)
    lse = torch.logsumexp(logits, dim=1)
    counts = target != IGNORE
    rows = torch.nonzero(counts)[:, 0]
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - logits[rows, target[rows]]
    lse = lse * counts
    if c["op"] == "loss":
        return {"loss": loss, "lse": lse}
    d = torch.zeros_like(logits)
    d[rows] = torch.softmax(logits[rows], dim=1)
    d[rows, target[rows]] -= 1.0
    d *= state["dloss"].double()[:, None]
    return {"loss": loss, "lse": lse, "dx": torch.einsum("tv,vh->th", d, w), "dw": torch.einsum("tv,th->vh", d, x)}
