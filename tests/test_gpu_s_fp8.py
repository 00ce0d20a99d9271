"""GPU: the 8-bit quantiser (bit for bit its definition in 64 bits) and the
block-scaled 8-bit product (against 64 bits, within the bound of its own
roundings): odd sizes, every tile and division of k, both formats, both kinds
of scales, strides and alignments, beta, NaN and infinity, other streams and
graphs."""
import numpy as np
import pytest

import mixed_precision_matmul_gb300 as mpg
from fp8_plain import HALF_STEP, blocks, quantize, sum_bound, widen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


def tdtype(name):
    import torch
    return {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16,
            "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[name]


def sample(m, n, seed, dtype="fp32"):
    """Values over many magnitudes, with blocks of zeros."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, n), generator=g) * torch.exp(2 * torch.randn((m, 1), generator=g))
    x *= torch.exp(torch.randn((1, n), generator=g))
    if m > 2:
        x[m // 2] = 0
    return x.to(tdtype(dtype))


def same(got, want):
    got, want = got.cpu().double().numpy(), np.asarray(want)
    assert got.shape == want.shape
    assert np.array_equal(got, want, equal_nan=True), float(np.mean(got != want))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 1000), (129, 127), (257, 384), (130, 16), (64, 131)])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_quantizer_is_its_definition(rows, cols, dtype, fmt, block):
    x = sample(rows, cols, rows * 7 + cols, dtype)
    size = 1 if block == "row" else 128
    q, s, qt, st = mpg.fp8_quantize(x.cuda(), fmt=fmt, block=block, transpose=True)
    wq, ws = quantize(x.double().numpy(), fmt, size)
    wqt, wst = quantize(x.double().numpy().T, fmt, size)
    same(s, ws)
    same(q, wq)
    same(st, wst)
    same(qt, wqt)
    q2, s2 = mpg.fp8_quantize(x.cuda(), fmt=fmt, block=block)
    same(s2, ws)
    same(q2, wq)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantizer_extremes(fmt):
    import torch
    top = 448.0 if fmt == "e4m3" else 57344.0
    x = torch.zeros((7, 300))
    x[0, 5] = 3.4e38
    x[1, 5] = 1e-44                                   # a subnormal maximum: the scale stays at 2^-126
    x[2, :] = top * 2.0 ** -7                         # exactly at the border of a power of two
    x[3, :] = float(np.nextafter(np.float32(top * 2.0 ** -7), np.float32(1e9)))
    x[4, 0], x[4, 1], x[4, 2] = float("inf"), 2.0, float("nan")
    x[5, 130:] = float("-inf")
    x[6, 0], x[6, 1] = -0.0, 1.0
    q, s, qt, st = mpg.fp8_quantize(x.cuda(), fmt=fmt, transpose=True)
    wq, ws = quantize(x.double().numpy(), fmt, 1)
    same(s, ws)
    same(q, wq)
    wqt, wst = quantize(x.double().numpy().T, fmt, 1)
    same(st, wst)
    same(qt, wqt)
    assert np.signbit(q.cpu().float().numpy()[6, 0])


def test_quantizer_strides_and_alignments():
    """Views that start off 16 bytes, padded lines, outputs at any address; only
    what belongs to the matrix is written."""
    import torch
    base = sample(70, 400, 5)
    for dt, off in (("fp32", 1), ("bf16", 3), ("fp16", 8)):
        x = base.to(tdtype(dt)).cuda()[3:, off:off + 290]
        q, s, qt, st = mpg.fp8_quantize(x, transpose=True)
        wq, ws = quantize(x.cpu().double().numpy(), "e4m3", 1)
        wqt, wst = quantize(x.cpu().double().numpy().T, "e4m3", 1)
        same(q, wq), same(s, ws), same(qt, wqt), same(st, wst)
    x = base.cuda().contiguous()
    for ldq, ldqt, o in ((400, 70, 0), (403, 77, 1), (416, 80, 3)):
        qb = torch.full((70 * ldq + 8,), 0x55, dtype=torch.uint8, device="cuda")
        tb = torch.full((400 * ldqt + 8,), 0x55, dtype=torch.uint8, device="cuda")
        s = torch.empty((70, 4), device="cuda")
        st = torch.empty((400, 1), device="cuda")
        mpg.fp8_quantize_raw(70, 400, x.data_ptr(), 400, mpg.F32, mpg.E4M3, 1, qb.data_ptr() + o, ldq, s.data_ptr(), 4, 1,
                             tb.data_ptr() + o, ldqt, st.data_ptr(), 1, 1)
        torch.cuda.synchronize()
        q = qb[o:o + 70 * ldq].view(70, ldq)
        t = tb[o:o + 400 * ldqt].view(400, ldqt)
        same(q[:, :400].contiguous().view(torch.float8_e4m3fn), quantize(base.double().numpy(), "e4m3", 1)[0])
        same(t[:, :70].contiguous().view(torch.float8_e4m3fn), quantize(base.double().numpy().T, "e4m3", 1)[0])
        assert (q[:, 400:] == 0x55).all() and (t[:, 70:] == 0x55).all()
        assert (qb[:o] == 0x55).all() and (qb[o + 70 * ldq:] == 0x55).all()
    # the transposed form alone
    st2 = torch.empty((400, 1), device="cuda")
    t2 = torch.empty((400, 70), dtype=torch.uint8, device="cuda")
    mpg.fp8_quantize_raw(70, 400, x.data_ptr(), 400, mpg.F32, mpg.E4M3, 1, 0, 0, 0, 0, 0, t2.data_ptr(), 70,
                         st2.data_ptr(), 1, 1)
    same(t2.view(torch.float8_e4m3fn), quantize(base.double().numpy().T, "e4m3", 1)[0])


def operand(rows, k, seed, fmt="e4m3", size=1, free=False):
    """Random codes (every finite value occurs) and scales; (codes, scales) on the CPU."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, k), generator=g) * (60.0 if fmt == "e4m3" else 3000.0)
    t = x.clamp(-448, 448).to(tdtype(fmt)) if fmt == "e4m3" else x.to(tdtype(fmt))
    s = torch.exp(torch.randn((-(-rows // size), blocks(k)), generator=g))
    if not free:
        s = torch.exp2(torch.round(torch.log2(s)))
    return t, s


def check(m, n, k, fmts=("e4m3", "e4m3"), sizes=(1, 128), out="fp32", opts=None, alpha=1.0, beta=0.0, seed=0,
          layout=None):
    import torch
    a, sa = operand(m, k, 2 * seed + 1, fmts[0], sizes[0], free=True)
    b, sb = operand(n, k, 2 * seed + 2, fmts[1], sizes[1], free=seed % 2 == 0)
    A, SA, B, SB = a.cuda(), sa.cuda(), b.cuda(), sb.cuda()
    if layout:
        A, SA, B, SB = layout(A, SA, B, SB)
    c0 = torch.randn((m, n), generator=torch.Generator().manual_seed(seed)).to(tdtype(out))
    C = c0.cuda()
    r = mpg.gemm_fp8(A, SA, B, SB, C=C, alpha=alpha, beta=beta, opts=mpg.options(**opts) if opts else None)
    assert r is C
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK
    wa = widen(a.double().numpy(), sa.double().numpy(), sizes[0])
    wb = widen(b.double().numpy(), sb.double().numpy(), sizes[1])
    want = alpha * (wa @ wb.T) + beta * c0.double().numpy()
    den = abs(alpha) * (np.abs(wa) @ np.abs(wb).T) + abs(beta) * np.abs(c0.double().numpy())
    got = C.cpu().double().numpy()
    err = np.abs(got - want)
    bound = sum_bound(k) * den + HALF_STEP[out] * np.abs(want) * (1 + 1e-3)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-300)))
    return C


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 128, 128), (1, 1000, 777), (2, 17, 300), (5, 384, 1024), (16, 257, 640), (17, 129, 4096),
    (33, 640, 2000), (64, 200, 1408), (65, 300, 513), (128, 128, 256), (130, 259, 129), (300, 1, 400), (257, 520, 2048),
])
def test_product_sizes(m, n, k):
    check(m, n, k, seed=m)


@pytest.mark.parametrize("fmts", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("sizes", [(1, 1), (1, 128), (128, 1), (128, 128)])
@pytest.mark.parametrize("m", [7, 140])
def test_product_formats_and_scales(fmts, sizes, m):
    check(m, 270, 500, fmts, sizes, seed=m + 1)


@pytest.mark.parametrize("tile", [16, 32, 64, 128])
@pytest.mark.parametrize("splits", [1, 2, 3, 5, 8])
def test_product_tiles_and_ranges(tile, splits):
    """Every tile on more rows than it holds, every division of k, one that leaves no block for the last range."""
    check(90, 200, 9 * 128 + 5, opts=dict(tile_n=tile, splitk=splits), seed=tile + splits)
    check(90, 200, 200, sizes=(1, 1), opts=dict(tile_n=tile, splitk=splits), seed=tile + splits)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (100, 300, 130), (256, 256, 128), (257, 255, 640), (513, 700, 1500),
                                   (300, 129, 128 * 40 + 16)])
@pytest.mark.parametrize("sizes", [(1, 128), (1, 1), (128, 128)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_product_on_pairs(m, n, k, sizes, out):
    check(m, n, k, sizes=sizes, out=out, opts=dict(cta_pair=1), alpha=0.5, beta=0.25 if m == 513 else 0.0, seed=m)


def test_product_on_pairs_many_tiles():
    """More tiles than clusters, each cluster several, and formats that differ."""
    check(2500, 2600, 300, ("e5m2", "e4m3"), (1, 1), opts=dict(cta_pair=1), seed=3)
    check(2500, 2600, 400, ("e4m3", "e4m3"), (1, 128), out="bf16", seed=4)


@pytest.mark.parametrize("m,n,k", [(2500, 2600, 300), (2433, 2561, 900)])
@pytest.mark.parametrize("fmts,sizes,out", [(("e5m2", "e4m3"), (1, 1), "fp32"), (("e4m3", "e4m3"), (1, 128), "bf16")])
def test_product_tile_after_tile(m, n, k, fmts, sizes, out):
    """More 128 x 128 tiles than SMs, each CTA several; lines of C on and off the vectors' alignment; beta."""
    check(m, n, k, fmts, sizes, out=out, opts=dict(cta_pair=-1), alpha=0.5, beta=-0.5 if m == 2433 else 0.0, seed=m)


@pytest.mark.parametrize("m", [3, 150])
@pytest.mark.parametrize("out", ["fp32", "fp16", "bf16"])
def test_product_outputs_alpha_beta(m, out):
    check(m, 136, 300, out=out, alpha=1e-3, beta=-0.75, seed=4)
    check(m, 135, 300, out=out, alpha=-1e-3, beta=0.0, seed=5)


@pytest.mark.parametrize("m", [2, 160])
def test_product_long_k_in_ring(m):
    """More blocks of k than stages, accumulator buffers and scale slots hold, many times over."""
    check(m, 130, 128 * 67 + 64, opts=dict(splitk=1), seed=6)


@pytest.mark.parametrize("m", [1, 20, 140])
def test_product_strides_and_alignments(m):
    import torch

    def padded(t, ld, off):
        base = torch.empty(t.shape[0] * ld + 64, dtype=torch.uint8, device="cuda").fill_(0x7E)
        v = base[off:off + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
        v.copy_(t.view(torch.uint8))
        return v.view(t.dtype)

    def f(ld, off):
        def g(A, SA, B, SB):
            # scales block by block and spread out
            sa = torch.full((SA.shape[1], 2 * SA.shape[0]), float("nan"), device="cuda")
            sa[:, ::2] = SA.t()
            return padded(A, ld, off), sa[:, ::2].t(), padded(B, ld + 16, off), SB.t().contiguous().t()
        return g
    for k, ld, off in ((300, 304, 0), (300, 320, 16), (300, 300, 0), (300, 307, 0), (300, 304, 1), (299, 301, 7)):
        check(m, 150, k, layout=f(ld, off), seed=k + ld)


def test_product_stores_nothing_beyond_c():
    import torch
    for m in (3, 140):
        a, sa = operand(m, 256, 1)
        b, sb = operand(135, 256, 2)
        buf = torch.full((m + 2, 150), 7.0, device="cuda")
        C = buf[1:m + 1, 5:140]
        mpg.gemm_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), C=C)
        C.fill_(7.0)
        assert (buf == 7.0).all()


def test_product_degenerate():
    import torch
    C = torch.full((3, 4), 2.0, device="cuda")
    e = torch.empty((3, 0), dtype=torch.float8_e4m3fn, device="cuda")
    f = torch.empty((4, 0), dtype=torch.float8_e4m3fn, device="cuda")
    z = torch.empty((3, 0), device="cuda"), torch.empty((4, 0), device="cuda")
    mpg.gemm_fp8(e, z[0], f, z[1], C=C, beta=0.5)
    assert (C == 1.0).all()
    a, sa = operand(3, 256, 1)
    b, sb = operand(4, 256, 2)
    mpg.gemm_fp8(a.cuda(), sa.cuda() * float("nan"), b.cuda(), sb.cuda(), C=C, alpha=0.0, beta=3.0)
    assert (C == 3.0).all()
    assert mpg.gemm_fp8(a.cuda()[:0], sa.cuda()[:0], b.cuda(), sb.cuda()).shape == (0, 4)
    # beta = 0 does not read C
    C.fill_(float("nan"))
    mpg.gemm_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), C=C)
    assert torch.isfinite(C).all()


@pytest.mark.parametrize("m", [4, 150])
def test_product_nan_stays_in_its_row_and_column(m):
    import torch
    n, k = 200, 384
    a, sa = operand(m, k, 1)
    b, sb = operand(n, k, 2, size=1)
    a.view(torch.uint8)[1, 130] = 0x7F                     # e4m3's NaN
    sb[3, 1] = float("nan")
    sa[2, 0] = float("inf")
    C = mpg.gemm_fp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=torch.float32).cpu()
    bad = ~torch.isfinite(C)
    want = torch.zeros((m, n), dtype=torch.bool)
    want[1] = want[2] = True
    want[:, 3] = True
    assert torch.equal(bad, want)


def test_product_repeats_bit_for_bit_and_on_other_streams():
    import torch
    for m, n, k in ((1, 4096, 4096), (40, 1000, 4096), (200, 300, 4096), (700, 900, 1000)):
        a, sa = operand(m, k, 1)
        b, sb = operand(n, k, 2, size=128)
        args = [t.cuda() for t in (a, sa, b, sb)]
        first = mpg.gemm_fp8(*args)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        outs = [mpg.gemm_fp8(*args) for _ in range(5)] + [mpg.gemm_fp8(*args, stream=side) for _ in range(5)]
        torch.cuda.synchronize()
        assert all(torch.equal(first, o) for o in outs)


def test_quantize_and_product_in_a_graph():
    import torch
    x = sample(33, 520, 3).cuda()
    w = sample(200, 520, 4).cuda()
    wq, ws = mpg.fp8_quantize(w, block="tile")
    y0 = mpg.gemm_fp8(*mpg.fp8_quantize(x), wq, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        y = mpg.gemm_fp8(*mpg.fp8_quantize(x), wq, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y0)
    x.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.float(), 2 * y0.float())


def test_linear_layer_gradients():
    """The three products of a layer and their gradients: each against the
    formula on the quantised values, and the gradient of the input against
    differences of the loss along random directions."""
    import torch
    m, n, k = 200, 260, 390
    g = torch.Generator().manual_seed(9)
    x, w = torch.randn((m, k), generator=g), torch.randn((n, k), generator=g) / k ** 0.5
    dy = torch.randn((m, n), generator=g)
    xq, xs, xqt, xst = mpg.fp8_quantize(x.cuda(), transpose=True)
    wq, ws, wqt, wst = mpg.fp8_quantize(w.cuda(), block="tile", transpose=True)
    dq, ds, dqt, dst = mpg.fp8_quantize(dy.cuda(), fmt="e5m2", transpose=True)
    f32 = torch.float32
    y = mpg.gemm_fp8(xq, xs, wq, ws, out_dtype=f32).cpu().double().numpy()
    dx = mpg.gemm_fp8(dq, ds, wqt, wst, out_dtype=f32).cpu().double().numpy()
    dw = mpg.gemm_fp8(dqt, dst, xqt, xst, out_dtype=f32).cpu().double().numpy()

    def w64(q, s, size):
        return widen(q.cpu().double().numpy(), s.cpu().double().numpy(), size)
    X, W, D = w64(xq, xs, 1), w64(wq, ws, 128), w64(dq, ds, 1)
    Dt, Xt, Wt = w64(dqt, dst, 1), w64(xqt, xst, 1), w64(wqt, wst, 128)
    assert np.array_equal(Wt, W.T)
    for got, p, r, depth in ((y, X, W.T, k), (dx, D, Wt.T, n), (dw, Dt, Xt.T, m)):
        den = np.abs(p) @ np.abs(r)
        assert np.all(np.abs(got - p @ r) <= (sum_bound(depth) + 2.0 ** -24) * den)
    # loss = sum(D * (X W^T)): its difference along V is sum(dx * V), X enters linearly
    V = np.random.Generator(np.random.PCG64(1)).standard_normal((m, k))
    h = 2.0 ** -10
    diff = (np.sum(D * ((X + h * V) @ W.T)) - np.sum(D * ((X - h * V) @ W.T))) / (2 * h)
    den = np.sum(np.abs(D) @ np.abs(W) * np.abs(V))
    assert abs(diff - np.sum(dx * V)) <= (sum_bound(n) + 2.0 ** -24) * den
