"""The operators of a low-precision training step, as measured cases: the quantiser to 8 bits with a scale for each block of 128,
the 8-bit product on such blocks, and the orthogonalised update.

``run`` computes them in plain torch where ``own`` is false (32-bit sums, rounded once at the end) and through the library's entry
points where it is true.  ``exact`` gives the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

BLOCK = 128
#: largest finite value of each 8-bit type, as 0.875 * 2**e
TOP_EXP = {"e4m3": 9, "e5m2": 16}
EIGHT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
#: the quintic whose five steps carry every singular value of a normalised matrix near 1
COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token's hidden vector on its way into an 8-bit layer while serving: latency
        {"name": "quantize token", "op": "quantize", "rows": 1, "cols": 8192, "dtype": "bf16", "fmt": "e4m3", "block": "row", "transpose": False},
        # activations of a training step, for the product and (transposed) for the weight gradient; a ragged token count
        {"name": "quantize activations", "op": "quantize", "rows": 8190, "cols": 8192, "dtype": "bf16", "fmt": "e4m3", "block": "row", "transpose": True},
        # output gradients in the wider 8-bit type, odd sizes on both sides
        {"name": "quantize gradients odd", "op": "quantize", "rows": 1531, "cols": 4100, "dtype": "fp16", "fmt": "e5m2", "block": "row", "transpose": True},
        # master weights after an optimiser step, in 128 x 128 blocks, for the forward product and the input gradient
        {"name": "quantize weights", "op": "quantize", "rows": 4096, "cols": 11008, "dtype": "fp32", "fmt": "e4m3", "block": "tile", "transpose": True},
        # one token through a layer while serving: the weights' bytes
        {"name": "product one token", "op": "product", "m": 1, "n": 8192, "k": 8192, "a_fmt": "e4m3", "b_fmt": "e4m3", "b_block": "tile", "out": "bf16"},
        # a batch of tokens being decoded, with k that ends inside a block
        {"name": "product 33 tokens", "op": "product", "m": 33, "n": 4096, "k": 4160, "a_fmt": "e4m3", "b_fmt": "e4m3", "b_block": "tile", "out": "fp16"},
        # a ragged prompt: every side ends inside a tile, and lines that are no multiple of 16 bytes
        {"name": "product ragged", "op": "product", "m": 1000, "n": 1531, "k": 4099, "a_fmt": "e4m3", "b_fmt": "e4m3", "b_block": "tile", "out": "bf16"},
        # weight gradient of a layer over 4096 tokens: scales along the tokens on both sides, fp32 out, gradients in e5m2
        {"name": "product weight gradient", "op": "product", "m": 4096, "n": 4096, "k": 4096, "a_fmt": "e5m2", "b_fmt": "e4m3", "b_block": "row", "out": "fp32"},
        # the forward product of a large layer in training
        {"name": "product 8192", "op": "product", "m": 8192, "n": 8192, "k": 8192, "a_fmt": "e4m3", "b_fmt": "e4m3", "b_block": "tile", "out": "bf16"},
        # the update of one small matrix: latency
        {"name": "orthogonalize small", "op": "orthogonalize", "batch": 1, "rows": 256, "cols": 1000, "dtype": "bf16", "steps": 5},
        # the matrices of twelve layers of one shape, taller than wide
        {"name": "orthogonalize layers", "op": "orthogonalize", "batch": 12, "rows": 2048, "cols": 768, "dtype": "fp32", "steps": 5},
        # one large layer's update
        {"name": "orthogonalize 4096", "op": "orthogonalize", "batch": 1, "rows": 4096, "cols": 4096, "dtype": "bf16", "steps": 5},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _pick(rng, low, high):
    """As _spread; one time in two a multiple of 128 where the range has one."""
    v = _spread(rng, low, high)
    if rng.random() < 0.5 and high >= 128:
        v = min(high // 128 * 128, max(128, v // 128 * 128))
    return v


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "orthogonalize"])
    if op == "quantize":
        rows = _spread(rng, 1, 16384)
        cols = _pick(rng, 128, min(16384, 8190 * 8192 // rows))
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["fp32", "fp16", "bf16"]), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "block": rng.choice(["row", "row", "tile"]), "transpose": rng.random() < 0.5}
    if op == "product":
        n, k = _pick(rng, 256, 16384), _pick(rng, 128, 16384)
        m = _spread(rng, 1, min(16384, 8192 ** 3 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "a_fmt": rng.choice(["e4m3", "e4m3", "e5m2"]), "b_fmt": "e4m3",
                "b_block": rng.choice(["tile", "tile", "row"]), "out": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    rows, cols = _pick(rng, 64, 4096), _pick(rng, 64, 4096)
    one = min(rows, cols) ** 2 * max(rows, cols)
    batch = _spread(rng, 1, max(1, min(24, 4096 ** 3 // one)))
    return {"op": op, "batch": batch, "rows": rows, "cols": cols, "dtype": rng.choice(["fp32", "bf16"]), "steps": 5}


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    c = case
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    if c["op"] == "quantize":
        r, n = c["rows"], c["cols"]
        forms = 2 if c["transpose"] else 1
        if c["block"] == "row":
            scales = r * _blocks(n) + (n * _blocks(r) if c["transpose"] else 0)
        else:
            scales = forms * _blocks(r) * _blocks(n)
        return {"bytes": r * n * (size[c["dtype"]] + forms) + 4 * scales, "flops": 0}
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        scales = m * _blocks(k) + (n if c["b_block"] == "row" else _blocks(n)) * _blocks(k)
        return {"bytes": m * k + n * k + 4 * scales + m * n * size[c["out"]], "flops": 2 * m * n * k}
    m, n = sorted((c["rows"], c["cols"]))
    # the two symmetric products need half of their elements
    flops = c["steps"] * (m * m * n + m * m * m + 2 * m * m * n)
    return {"bytes": c["batch"] * m * n * (size[c["dtype"]] + 2), "flops": c["batch"] * flops}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _split_scale(amax, fmt):
    """The power of two that carries amax under the type's largest value (1 for an empty block)."""
    f, e = torch.frexp(amax)
    t = (e - TOP_EXP[fmt] + (f > 0.875).to(e.dtype)).clamp(min=-126)
    power = ((t.to(torch.int32) + 127) << 23).view(torch.float32)      # 2**t exactly
    return torch.where(amax > 0, power, 1.0)


def _padded(x, rows, cols):
    """x with zeros up to whole blocks of (rows, cols)."""
    m, n = x.shape
    return torch.nn.functional.pad(x, (0, -n % cols, 0, -m % rows))


def _quantize(x, fmt, rows):
    """(8-bit values, scales) with one scale for each block of `rows` x 128: the plain form of the quantiser."""
    m, n = x.shape
    p = _padded(x.float(), rows, BLOCK)
    b = p.view(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)
    s = _split_scale(torch.where(b.isfinite(), b.abs(), 0).amax(dim=(1, 3)), fmt)
    q = (b / s[:, None, :, None]).view(p.shape)[:m, :n].to(EIGHT[fmt])
    return q.contiguous(), s


def _free_scales(x, rows):
    """e4m3 values with a scale of amax / 448 for each block, as weights are stored that were quantised elsewhere."""
    m, n = x.shape
    p = _padded(x.float(), rows, BLOCK)
    b = p.view(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)
    s = b.abs().amax(dim=(1, 3)).clamp(min=1e-12) / 448.0
    return (b / s[:, None, :, None]).view(p.shape)[:m, :n].to(EIGHT["e4m3"]).contiguous(), s.contiguous()


def _activations(m, n, g, dev):
    """Normal values with a few channels that are much larger than the others, as hidden states have them."""
    channel = torch.exp(0.5 * torch.randn(n, generator=g, device=dev)) * torch.where(torch.rand(n, generator=g, device=dev) < 0.004, 20.0, 1.0)
    return torch.randn((m, n), generator=g, device=dev) * channel


def _gradients(m, n, g, dev):
    """Small values whose size differs from token to token."""
    return torch.randn((m, n), generator=g, device=dev) * (1e-4 * torch.exp(torch.randn((m, 1), generator=g, device=dev)))


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    if c["op"] == "quantize":
        make = _gradients if c["fmt"] == "e5m2" else _activations
        return {"case": c, "x": make(c["rows"], c["cols"], g, dev).to(TYPES[c["dtype"]])}
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        make = _gradients if c["a_fmt"] == "e5m2" else _activations
        a, sa = _quantize(make(m, k, g, dev), c["a_fmt"], 1)
        if c["b_block"] == "row":
            b, sb = _quantize(_activations(n, k, g, dev), c["b_fmt"], 1)
        else:
            b, sb = _free_scales(0.02 * torch.randn((n, k), generator=g, device=dev), BLOCK)
        # scales of single rows lie block by block, as the quantiser lays them
        sa = sa.t().contiguous().t()
        sb = sb.t().contiguous().t() if c["b_block"] == "row" else sb
        return {"case": c, "a": a, "sa": sa, "b": b, "sb": sb}
    # the momentum of a weight gradient: a few strong directions over noise
    b, m, n = c["batch"], c["rows"], c["cols"]
    r = max(4, min(m, n) // 32)
    strong = torch.randn((b, m, r), generator=g, device=dev) @ torch.randn((b, r, n), generator=g, device=dev)
    x = 1e-3 * (torch.randn((b, m, n), generator=g, device=dev) + strong / math.sqrt(r))
    return {"case": c, "g": x.to(TYPES[c["dtype"]])}


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def _wide(q, s):
    """The fp32 values that 8-bit values and their scales stand for."""
    m, n = q.shape
    rows = 1 if s.shape[0] == m else BLOCK
    s = s.repeat_interleave(BLOCK, dim=1)[:, :n]
    s = s if rows == 1 else s.repeat_interleave(BLOCK, dim=0)[:m]
    return q.float() * s


def _plain(state):
    c = state["case"]
    if c["op"] == "quantize":
        rows = 1 if c["block"] == "row" else BLOCK
        q, s = _quantize(state["x"], c["fmt"], rows)
        if not c["transpose"]:
            return {"q": q, "s": s}
        qt, st = _quantize(state["x"].t(), c["fmt"], rows)
        return {"q": q, "s": s, "qt": qt, "st": st}
    if c["op"] == "product":
        return _wide(state["a"], state["sa"]).matmul(_wide(state["b"], state["sb"]).t()).to(TYPES[c["out"]])
    x = state["g"].float()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    a, b, cc = COEFFS
    for _ in range(c["steps"]):      # the steps follow from one another
        s = x @ x.mT
        x = a * x + (b * s + cc * (s @ s)) @ x
    return (x.mT if tall else x).to(torch.bfloat16).contiguous()


def _own(state):
    import mixed_precision_matmul_gb300 as mpg
    c = state["case"]
    if c["op"] == "quantize":
        r = mpg.fp8_quantize(state["x"], fmt=c["fmt"], block=c["block"], transpose=c["transpose"])
        return dict(zip(("q", "s", "qt", "st"), r))
    if c["op"] == "product":
        return mpg.gemm_fp8(state["a"], state["sa"], state["b"], state["sb"], out_dtype=TYPES[c["out"]])
    return mpg.orthogonalize(state["g"], steps=c["steps"], coeffs=COEFFS, eps=EPS)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _two_to(t):
    """2**t in 64 bits, exactly (t whole, within the normal range)."""
    return ((t.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quantize(x, fmt, block):
    """Block maxima by segments of the flattened index, powers of two from the logarithm's neighbours, rounding to the 8-bit grid."""
    top = 0.875 * 2.0 ** TOP_EXP[fmt]
    mantissa, lowest = {"e4m3": (3, -6), "e5m2": (2, -14)}[fmt]
    m, n = x.shape
    tall = BLOCK if block == "tile" else 1
    rb = torch.arange(m, device=x.device) // tall
    cb = torch.arange(n, device=x.device) // BLOCK
    shape = (int(rb[-1]) + 1, int(cb[-1]) + 1)
    # maxima over columns' blocks, then over rows' blocks
    part = torch.zeros((m, shape[1]), dtype=torch.float64, device=x.device).scatter_reduce_(1, cb.expand(m, n), x.abs(), "amax")
    amax = torch.zeros(shape, dtype=torch.float64, device=x.device).scatter_reduce_(0, rb[:, None].expand(m, shape[1]), part, "amax")
    t = torch.floor(torch.log2(torch.where(amax > 0, amax, top) / top)) - 1
    for _ in range(3):               # the smallest power of two that is large enough
        t = torch.where(amax > top * _two_to(t), t + 1, t)
    s = torch.where(amax > 0, _two_to(t.clamp(min=-126)), 1.0)
    v = x / s[rb][:, cb]
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** (lowest - 1)))).clamp(min=lowest)
    e = torch.where(v.abs() >= _two_to(e + 1), e + 1, torch.where((v.abs() < _two_to(e)) & (e > lowest), e - 1, e))
    step = _two_to(e - mantissa)
    return torch.round(v / step) * step, s


def exact(case, seed):
    c = case
    state = prepare(case, seed)
    if c["op"] == "quantize":
        x = state["x"].double()
        q, s = _exact_quantize(x, c["fmt"], c["block"])
        if not c["transpose"]:
            return {"q": q, "s": s}
        qt, st = _exact_quantize(x.t(), c["fmt"], c["block"])
        return {"q": q, "s": s, "qt": qt, "st": st}
    if c["op"] == "product":
        def index(s, n):
            return torch.arange(n, device=s.device) // (1 if s.shape[0] == n else BLOCK)
        m, n, k = c["m"], c["n"], c["k"]
        kb = torch.arange(k, device="cuda") // BLOCK
        a = state["a"].double() * state["sa"].double()[index(state["sa"], m)][:, kb]
        b = state["b"].double() * state["sb"].double()[index(state["sb"], n)][:, kb]
        return torch.einsum("ik,jk->ij", a, b)
    if work(case)["flops"] > 1.2e13:     # over about 20 seconds in 64 bits
        return None
    y = state["g"].double()
    wide = y.shape[2] > y.shape[1]
    y = y.transpose(1, 2) if wide else y
    y = y / (torch.linalg.matrix_norm(y)[:, None, None] + EPS)
    one = torch.eye(y.shape[2], dtype=y.dtype, device=y.device)
    for _ in range(c["steps"]):
        s = y.transpose(1, 2) @ y
        y = y @ (COEFFS[0] * one + s @ (COEFFS[1] * one + COEFFS[2] * s))
    return (y.transpose(1, 2) if wide else y).contiguous()
