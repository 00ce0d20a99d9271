"""GPU: the orthogonalised update against 64 bits.  One step is held to a bound
element by element that counts its roundings; several steps to twice the error
of the same roundings made in plain torch; and the singular values of the
result to what the polynomial does to them."""
import math

import numpy as np
import pytest

import mixed_precision_matmul_gb300 as mpg

pytestmark = pytest.mark.gpu

HALF_STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
A, B, C = mpg.NS_COEFFS


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


def tdtype(name):
    import torch
    return {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[name]


def momentum(b, m, n, seed, dtype):
    import torch
    g = torch.Generator().manual_seed(seed)
    r = max(1, min(m, n) // 16)
    x = torch.randn((b, m, n), generator=g)
    x += torch.randn((b, m, r), generator=g) @ torch.randn((b, r, n), generator=g) / math.sqrt(r)
    return (1e-3 * x).to(tdtype(dtype))


def exact(g, steps, eps=1e-7):
    """Wide or tall, S on the shorter side, in 64 bits."""
    x = g.double()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + eps)
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    for _ in range(steps):
        s = x @ x.mT
        x = A * x + (B * s + C * (s @ s)) @ x
    return x.mT if tall else x


def rounded(g, steps, eps=1e-7):
    """The same with every stored matrix rounded to fp16 (sums in fp32): what the
    operator's choice of storage costs."""
    def f16(x):
        return x.half().float()
    x = g.float()
    norm = x.double().square().sum(dim=(1, 2), keepdim=True).sqrt().float()
    scale = 2.0 ** round(math.log2(math.sqrt(max(x.shape[1:]))))
    e = 2.0 ** (-math.floor(math.log2(float(norm[0]) / math.sqrt(x.shape[1] * x.shape[2]))))
    x, f = f16(x * e), 1 / ((norm + eps) * e)
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    for i in range(steps):
        s = f16((x @ x.mT) * f * f)
        y = (A * x + f16(B * s + C * (s @ s)) @ x) * f
        x, f = f16(y * scale), 1 / scale
    return y.mT if tall else y


@pytest.mark.parametrize("b,m,n", [(1, 1, 1), (1, 1, 300), (2, 300, 1), (3, 5, 7), (1, 128, 128), (1, 129, 257),
                                   (2, 64, 500), (2, 500, 64), (1, 300, 258), (1, 260, 515)])
@pytest.mark.parametrize("dtype,out", [("bf16", "fp32"), ("fp16", "bf16"), ("fp32", "fp16")])
def test_one_step_within_its_roundings(b, m, n, dtype, out):
    import torch
    g = momentum(b, m, n, m + n, dtype)
    got = mpg.orthogonalize(g.cuda(), steps=1, out_dtype=tdtype(out)).cpu().double()
    assert mpg.device_status() == mpg.OK
    want = exact(g, 1)
    u = 2.0 ** -11                                    # half a step of fp16
    tiny = 2.0 ** -25                                 # and below its normal range
    x = g.double()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + 1e-7)
    tall = m > n
    x = (x.mT if tall else x)
    # fp32 gradients are rounded on their way in; tensor-core sums are off by a step of fp32 a term
    dx = x.abs() * ((u if dtype == "fp32" else 0.0) + 2.0 ** -20)

    def product(p, dp, r, dr):
        return dp @ r.abs() + p.abs() @ dr + dp @ dr + p.shape[2] * 2.0 ** -23 * ((p.abs() + dp) @ (r.abs() + dr))
    s = x @ x.mT
    ds = product(x, dx, x.mT, dx.mT)
    ds = ds + u * (s.abs() + ds) + tiny
    p = B * s + C * (s @ s)
    dp = abs(B) * ds + abs(C) * product(s, ds, s, ds) + 2.0 ** -22 * (abs(B) * s.abs() + abs(C) * (s.abs() @ s.abs()))
    dp = dp + u * (p.abs() + dp) + tiny
    d = product(p, dp, x, dx) + A * dx + 2.0 ** -21 * (A * x.abs() + p.abs() @ x.abs())
    d = d.mT if tall else d
    bound = d + (want.abs() + d) * HALF_STEP[out] + (2.0 ** -25 if out == "fp16" else 0.0)
    err = (got - want).abs()
    assert torch.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("b,m,n,dtype", [
    (1, 7, 3, "bf16"), (1, 100, 100, "fp32"), (2, 128, 512, "bf16"), (1, 513, 130, "fp16"), (3, 257, 300, "bf16"),
    (1, 256, 1000, "bf16"), (2, 768, 500, "fp32"), (1, 1030, 1025, "bf16"), (20, 520, 260, "bf16"),
    (76, 256, 256, "bf16"),                            # enough tiles for pairs of CTAs
    (10, 700, 900, "fp32"),
    (1, 100, 576, "bf16"),                             # 9 blocks of 64: a division that leaves the last range empty
    (1, 384, 1100, "bf16"), (1, 260, 2000, "fp16"),
])
def test_five_steps(b, m, n, dtype):
    g = momentum(b, m, n, m * 3 + n, dtype)
    got = mpg.orthogonalize(g.cuda(), out_dtype=tdtype("fp32")).cpu().double()
    assert mpg.device_status() == mpg.OK
    want, sim = exact(g, 5), rounded(g, 5).double()
    norm = want.flatten(1).norm(dim=1)
    predicted = ((sim - want).flatten(1).norm(dim=1) / norm).max()
    off = ((got - want).flatten(1).norm(dim=1) / norm).max()
    assert off <= 2 * predicted + 1e-5, (float(off), float(predicted))
    low = mpg.orthogonalize(g.cuda()).cpu().double()       # bf16: the same, rounded once more
    off = ((low - want).flatten(1).norm(dim=1) / norm).max()
    assert off <= 2 * predicted + HALF_STEP["bf16"]


def test_singular_values():
    import torch
    g = momentum(1, 200, 600, 1, "fp32")
    got = mpg.orthogonalize(g.cuda(), out_dtype=torch.float32).cpu().double()
    sv = torch.linalg.svdvals(got[0])
    p = torch.linalg.svdvals(g[0].double() / g[0].double().norm())
    for _ in range(5):
        p = A * p + B * p ** 3 + C * p ** 5
    assert float((sv.sort()[0] - p.sort()[0]).abs().max()) < 0.02
    assert 0.6 < float(sv.min()) and float(sv.max()) < 1.25


def test_two_dimensional_and_given_output():
    import torch
    g = momentum(2, 90, 200, 3, "fp32").cuda()
    o = mpg.orthogonalize(g[0], out_dtype=torch.float32)
    assert o.shape == (90, 200) and torch.equal(o, mpg.orthogonalize(g, out_dtype=torch.float32)[0])
    w = torch.randn((2, 90, 200), device="cuda")
    w0 = w.clone()
    r = mpg.orthogonalize(g, O=w, alpha=-0.02, beta=0.9)
    assert r is w
    want = 0.9 * w0.double() - 0.02 * mpg.orthogonalize(g, out_dtype=torch.float32).double()
    # alpha is folded into the last product's factor: a few roundings of fp32
    assert float((w.double() - want).abs().max()) <= 2.0 ** -21 * float(w0.abs().max() + 0.1)
    g2 = g.clone()
    assert torch.equal(mpg.orthogonalize(g2, O=g2), mpg.orthogonalize(g, out_dtype=torch.float32))


def test_strides():
    import torch
    g = momentum(3, 70, 130, 5, "bf16").cuda()
    want = mpg.orthogonalize(g)
    for off, ld in ((0, 136), (1, 133), (3, 150)):
        buf = torch.zeros((3, 75, ld), dtype=g.dtype, device="cuda")
        v = buf[:, 2:72, off:off + 130]
        v.copy_(g)
        obuf = torch.full((3, 75, ld), 7.0, dtype=g.dtype, device="cuda")
        o = obuf[:, 2:72, off:off + 130]
        mpg.orthogonalize(v, O=o)
        assert torch.equal(o, want)
        o.fill_(7.0)
        assert (obuf == 7.0).all()
    assert torch.equal(mpg.orthogonalize(g[:1].expand(3, 70, 130))[2], want[0])
    with pytest.raises(ValueError):
        mpg.orthogonalize(g.mT)
    with pytest.raises(ValueError):
        mpg.orthogonalize(g, O=g[:1].expand(3, 70, 130))


def test_scales_of_the_input():
    """A power of two in the input changes nothing but eps; zeros stay zeros;
    huge and tiny values keep the norm finite."""
    import torch
    g = momentum(1, 100, 180, 6, "fp32").cuda()
    base = mpg.orthogonalize(g, eps=0.0, out_dtype=torch.float32)
    for e in (-60, -20, 3, 90):
        assert torch.equal(base, mpg.orthogonalize(g * 2.0 ** e, eps=0.0, out_dtype=torch.float32)), e
    z = torch.zeros((2, 40, 50), device="cuda")
    z[1] = torch.randn((40, 50), device="cuda")
    o = mpg.orthogonalize(z)
    assert (o[0] == 0).all() and torch.isfinite(o).all() and (o[1] != 0).any()
    one = torch.zeros((1, 300, 400), device="cuda")
    one[0, 17, 33] = -5.0                              # the whole norm in one entry
    o = mpg.orthogonalize(one, out_dtype=torch.float32)
    p = 1.0
    for _ in range(5):
        p = A * p + B * p ** 3 + C * p ** 5
    assert abs(float(o[0, 17, 33]) + p) < 0.01 and float(o.abs().sum()) == abs(float(o[0, 17, 33]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_stays_in_its_matrix(bad):
    import torch
    g = momentum(3, 60, 150, 7, "bf16").cuda()
    want = mpg.orthogonalize(g)
    g[1, 10, 20] = bad
    got = mpg.orthogonalize(g)
    assert torch.isnan(got[1]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_repeats_streams_and_graphs():
    import torch
    for shape in ((1, 300, 500), (30, 256, 300)):
        g = momentum(*shape, 8, "bf16").cuda()
        first = mpg.orthogonalize(g)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        outs = [mpg.orthogonalize(g) for _ in range(3)] + [mpg.orthogonalize(g, stream=side) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(first, o) for o in outs)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o = mpg.orthogonalize(g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, o)
