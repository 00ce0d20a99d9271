"""Plain 64-bit forms of the gated feed-forward product, the cross entropy of a
projection and gradient clipping, with bounds of what their kernels may be off.

A sum of k products on the tensor cores is off by at most (k / 16 + 4) 2^-23 of
the sum of the products' absolute values: each instruction adds 16 products and
the running sum, aligned to the largest and cut off there (one unit of 24 bits of
the largest, which is at most the sum of absolute values), and parts of a split
sum are added in fp32.  A rounding to a type t is off by at most eps(t) / 2 of the
value, or half of fp16's smallest number, 2^-25.
"""
import torch

F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126 if dtype == torch.float32 else 2.0 ** -126


def sum_error(k):
    return (k / 16 + 4) * 2.0 ** -23


def act(g, name):
    """(act(g), act'(g)) in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / 2 ** 0.5)
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / (2 * torch.pi) ** 0.5
    c = (2 / torch.pi) ** 0.5
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


#: |act'| <= 1.13 and |act''| <= 1.13 for all three (the largest: gelu_tanh's)
SLOPE = 1.13
#: what the activations and their slopes are off by themselves: exponentials and
#: reciprocals of single instructions (2^-22 of the value, and the argument's
#: rounding, 2^-24 of at most 100 where the result is not rounded away), a few
#: operations
ACT = 2.0 ** -17


def gated(x, wg, wu, name):
    """y and what is kept for the gradients, act(g) and u act'(g), in 64 bits, and bounds of each but for the final rounding."""
    x, wg, wu = x.to(F64), wg.to(F64), wu.to(F64)
    g, u = x @ wg.t(), x @ wu.t()
    e = sum_error(x.shape[1])
    eg, eu = e * (x.abs() @ wg.abs().t()), e * (x.abs() @ wu.abs().t())
    a, d = act(g, name)
    ea = SLOPE * eg + ACT * (a.abs() + 2.0 ** -10)
    eb = SLOPE * (u.abs() + eu) * eg + SLOPE * eu + ACT * u.abs()
    ey = (SLOPE * u.abs() + SLOPE * eu) * eg + a.abs() * eu + ACT * (a.abs() + 2.0 ** -10) * u.abs()
    return (a * u, a, u * d), (ey, ea, eb)


def kept_values(t):
    """The values of what is kept in 64 bits: fp16, or codes with 6 bits of exponent and 9 of fraction."""
    if t.dtype != torch.int16:
        return t.to(F64)
    c = t.to(torch.int32) & 0x7fff
    e, f = c >> 9, (c & 511).to(F64) / 512
    v = torch.where(e == 0, f * 2.0 ** -30, (1 + f) * torch.exp2(e.to(F64) - 31))
    v = torch.where(e == 63, torch.where(f == 0, torch.inf, torch.nan), v)
    return torch.where(t < 0, -v, v)


def check_kept(t, ref, bound):
    """What is kept is ref rounded once: half a step is 2^-11 of the value in fp16, 2^-10 in codes."""
    r, least = (2.0 ** -10, 2.0 ** -40) if t.dtype == torch.int16 else (2.0 ** -11, 2.0 ** -25)
    off = (kept_values(t) - ref).abs()
    assert bool((off <= bound * (1 + r) + r * ref.abs() + least).all())


def gated_gradients(dy, x, wg, wu, name, kept=None):
    """(dx, dwg, dwu) in 64 bits and bounds of each but for the final rounding."""
    dtype = x.dtype
    x, wg, wu, dy = x.to(F64), wg.to(F64), wu.to(F64), dy.to(F64)
    if kept is None:
        e = sum_error(x.shape[1])
        g, u = x @ wg.t(), x @ wu.t()
        eg, eu = e * (x.abs() @ wg.abs().t()), e * (x.abs() @ wu.abs().t())
        a, d = act(g, name)
        b = u * d
        ea, eb = SLOPE * eg + ACT * (a.abs() + 2.0 ** -10), SLOPE * (u.abs() + eu) * eg + SLOPE * eu + ACT * u.abs()
    else:
        a, b = (kept_values(t) for t in kept)
        ea, eb = ACT * a.abs(), ACT * b.abs()
    dg, du = dy * b, dy * a
    # one rounding of dg and du each, as operands; in fp16 with a scale that leaves
    # subnormals 2^-28 of the largest dy, whose halves are 2^-29
    r = half_step(dtype)
    floor = float(dy.abs().max()) * 2.0 ** -29 if dtype == torch.float16 and dy.numel() else 0.0
    edg = dy.abs() * eb + r * dg.abs() + floor
    edu = dy.abs() * ea + r * du.abs() + floor
    i, t = wg.shape[0], x.shape[0]
    dx = dg @ wg + du @ wu
    ex = edg @ wg.abs() + edu @ wu.abs() + sum_error(2 * i) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    dwg, dwu = dg.t() @ x, du.t() @ x
    ewg = edg.t() @ x.abs() + sum_error(t) * (dg.abs().t() @ x.abs())
    ewu = edu.t() @ x.abs() + sum_error(t) * (du.abs().t() @ x.abs())
    return (dx, dwg, dwu), (ex, ewg, ewu)


def loss(x, w, target, ignore=-100):
    """(loss, lse) in 64 bits and bounds of each but for the final rounding."""
    x, w = x.to(F64), w.to(F64)
    l = x @ w.t()
    el = (sum_error(x.shape[1]) * (x.abs() @ w.abs().t())).amax(dim=1)
    lse = torch.logsumexp(l, dim=1)
    counts = target != ignore
    at = torch.where(counts, target, 0).long()
    value = torch.where(counts, lse - l.gather(1, at[:, None])[:, 0], 0.0)
    # (sums of at most 1024 of k are added in fp32 on the way: no more than the bound of one sum)
    # terms: logits' errors, the logits in units of ln 2 and their differences
    # (2^-24 each of the largest logit), exponentials 2^-22, sums of at most 256 in a
    # row and 2^11 parts after them
    e = el + 3 * 2.0 ** -24 * l.abs().amax(dim=1) + 2.0 ** -22 + 20 * 2.0 ** -24 * (1 + lse.abs())
    zero = torch.zeros_like(e)
    return (value, torch.where(counts, lse, zero)), (torch.where(counts, 2 * e, zero), torch.where(counts, e, zero))


def loss_gradients(x, w, target, lse, dloss, ignore=-100):
    """(dx, dw) in 64 bits (from the given lse) and bounds of each but for the final rounding."""
    dtype = x.dtype
    x, w, lse = x.to(F64), w.to(F64), lse.to(F64)
    counts = target != ignore
    at = torch.where(counts, target, 0).long()
    dl = torch.where(counts, dloss.to(F64), 0.0)[:, None]
    l = x @ w.t()
    p = torch.exp(l - lse[:, None])
    el = sum_error(x.shape[1]) * (x.abs() @ w.abs().t()) + 2 * 2.0 ** -23 * (l.abs() + lse.abs()[:, None]) + 2.0 ** -22
    d = p.clone()
    d.scatter_add_(1, at[:, None], torch.full_like(p[:, :1], -1.0))
    r = half_step(dtype)
    floor = float(dl.abs().max()) * 2.0 ** -38 if dtype == torch.float16 and dl.numel() else 0.0
    ed = dl.abs() * (p * torch.expm1(el) + r * d.abs()) + floor * (dl != 0)
    d = d * dl
    v, t = w.shape[0], x.shape[0]
    pieces = 1 + v * t // 2 ** 28
    dx, dw = d @ w, d.t() @ x
    ex = ed @ w.abs() + (sum_error(v) + pieces * 2.0 ** -23) * (d.abs() @ w.abs())
    ew = ed.t() @ x.abs() + sum_error(t) * (d.abs().t() @ x.abs())
    return (dx, dw), (ex, ew)


def check(out, ref, bound, dtype=None):
    """out is ref rounded once to its type, within bound before that."""
    dtype = dtype or out.dtype
    r = half_step(dtype)
    ref, bound = ref.to(out.device), bound.to(out.device)
    allowed = bound * (1 + r) + r * ref.abs() + tiny(dtype)
    off = (out.to(F64) - ref).abs()
    bad = ~(off <= allowed)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / allowed).nan_to_num(9e9).max()):.3g} of the bound"
