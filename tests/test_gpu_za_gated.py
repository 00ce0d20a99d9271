"""GPU: the gated feed-forward product and its gradients against 64 bits."""
import threading

import pytest

import mixed_precision_matmul_gb300 as mpg

torch = pytest.importorskip("torch")
import fused_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def operands(t, h, i, dtype, seed=0, pad=0, shift=0, dev="cuda"):
    """x, wg, wu, dy with lines `pad` elements longer and bases `shift` elements off."""
    g = torch.Generator().manual_seed(seed)

    def make(rows, cols, scale):
        buf = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=TYPES[dtype], device=dev)
        m = buf[shift:].view(rows, cols + pad)[:, :cols]
        m.copy_((scale * torch.randn(rows, cols, generator=g)).to(TYPES[dtype]))
        return m
    return make(t, h, 1.0), make(i, h, h ** -0.5), make(i, h, h ** -0.5), make(t, i, 0.1)


def ok():
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK


SHAPES = [
    (1, 1, 1), (1, 64, 64), (3, 100, 33), (8, 513, 40), (9, 64, 1000), (16, 1000, 7), (17, 72, 129), (32, 520, 264),
    (33, 64, 64), (33, 1, 5), (40, 72, 40), (64, 100, 33), (127, 128, 65), (130, 65, 70), (257, 200, 129), (300, 1001, 131),
]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t,h,i", SHAPES)
def test_product(t, h, i, act):
    for dtype, pad, shift in (("bf16", 0, 0), ("fp16", 8, 8), ("bf16", 3, 1)):
        x, wg, wu, _ = operands(t, h, i, dtype, 1, pad, shift)
        (y, a, b), (ey, ea, eb) = plain.gated(x, wg, wu, act)
        out = mpg.gated_gemm(x, wg, wu, act=act)
        ok()
        plain.check(out, y, ey)
        out, kg, ku = mpg.gated_gemm(x, wg, wu, act=act, keep=True)
        ok()
        plain.check(out, y, ey)
        plain.check_kept(kg, a, ea)
        plain.check_kept(ku, b, eb)


@pytest.mark.parametrize("t,h,i,dtype", [(2048, 512, 4096, "bf16"), (1531, 520, 2741, "fp16"), (4100, 264, 1030, "bf16"),
                                         (200, 4000, 300, "bf16"), (40, 3999, 70, "fp16"), (600, 4096, 515, "bf16")])
def test_product_on_pairs(t, h, i, dtype):
    x, wg, wu, _ = operands(t, h, i, dtype, 2)
    (y, a, b), (ey, ea, eb) = plain.gated(x, wg, wu, "silu")
    out, kg, ku = mpg.gated_gemm(x, wg, wu, keep=True)
    ok()
    plain.check(out, y, ey)
    plain.check_kept(kg, a, ea)
    plain.check_kept(ku, b, eb)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t,h,i", SHAPES + [(40, 64, 4000), (5, 72, 11000), (700, 130, 520)])
def test_gradients(t, h, i, act):
    for dtype, pad, shift in (("fp16", 0, 0), ("bf16", 8, 8), ("fp16", 3, 1)):
        x, wg, wu, dy = operands(t, h, i, dtype, 3, pad, shift)
        _, g, u = mpg.gated_gemm(x, wg, wu, act=act, keep=True)
        for kept in (None, (g, u)):
            refs, bounds = plain.gated_gradients(dy, x, wg, wu, act, kept)
            outs = mpg.gated_gemm_backward(dy, x, wg, wu, act=act, kept=kept)
            ok()
            for o, r, b in zip(outs, refs, bounds):
                plain.check(o, r, b)


@pytest.mark.parametrize("t,h,i,dtype", [(2048, 512, 2000, "bf16"), (1500, 1032, 3000, "fp16"), (4200, 256, 1030, "bf16"),
                                         (200, 4000, 300, "fp16"), (40, 3999, 70, "bf16"), (600, 4096, 515, "fp16"),
                                         (40, 1001, 1100, "bf16"), (300, 1003, 1100, "fp16"), (1100, 1001, 130, "bf16")])
def test_gradients_on_pairs(t, h, i, dtype):
    x, wg, wu, dy = operands(t, h, i, dtype, 4)
    _, g, u = mpg.gated_gemm(x, wg, wu, keep=True)
    for kept in (None, (g, u)):
        refs, bounds = plain.gated_gradients(dy, x, wg, wu, "silu", kept)
        outs = mpg.gated_gemm_backward(dy, x, wg, wu, kept=kept)
        ok()
        for o, r, b in zip(outs, refs, bounds):
            plain.check(o, r, b)


def test_gradient_against_differences():
    """Along a direction: (f(x + s d) - f(x - s d)) / 2 s of f = sum(y dy) in 64 bits, within
    the gradient's own bound and what the third derivative leaves (s^2 times order 1)."""
    x, wg, wu, dy = operands(50, 72, 96, "bf16", 5)
    for act in ("silu", "gelu", "gelu_tanh"):
        refs, bounds = plain.gated_gradients(dy, x, wg, wu, act)
        outs = mpg.gated_gemm_backward(dy, x, wg, wu, act=act)
        ok()
        base = [t.double() for t in (x, wg, wu)]
        for k in range(3):
            d = torch.randn(base[k].shape, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
            s = 1e-5

            def f(step):
                a = [t + step * d if j == k else t for j, t in enumerate(base)]
                gate, up = a[0] @ a[1].t(), a[0] @ a[2].t()
                return float((plain.act(gate, act)[0] * up * dy.double()).sum())
            slope = (f(s) - f(-s)) / (2 * s)
            r = plain.half_step(torch.bfloat16)
            allowed = float(((bounds[k] + r * refs[k].abs()) * d.abs()).sum()) + 1e-6
            assert abs(float((outs[k].double() * d).sum()) - slope) <= allowed


def test_what_is_not_needed_is_not_made():
    x, wg, wu, dy = operands(70, 64, 96, "bf16", 6)
    full = mpg.gated_gemm_backward(dy, x, wg, wu)
    dx, a, b = mpg.gated_gemm_backward(dy, x, wg, wu, need_dw=False)
    assert a is None and b is None and torch.equal(dx, full[0])
    a, dwg, dwu = mpg.gated_gemm_backward(dy, x, wg, wu, need_dx=False)
    assert a is None and torch.equal(dwg, full[1]) and torch.equal(dwu, full[2])
    assert mpg.gated_gemm_backward(dy, x, wg, wu, need_dx=False, need_dw=False) == (None, None, None)


def test_small_and_large_gradients_in_fp16():
    """Gradients of 2^-20 .. and of fp16's largest values keep their precision: dgate and dup
    carry a power of two."""
    x, wg, wu, dy = operands(64, 128, 200, "fp16", 7)
    for scale in (2.0 ** -16, 2.0 ** 14):
        small = (dy.double() * scale).half()
        refs, bounds = plain.gated_gradients(small, x, wg, wu, "silu")
        outs = mpg.gated_gemm_backward(small, x, wg, wu)
        ok()
        for o, r, b in zip(outs, refs, bounds):
            keep = r.abs() < 60000
            plain.check(torch.where(keep, o, 0), torch.where(keep, r, 0), b)
    zero = mpg.gated_gemm_backward(torch.zeros_like(dy), x, wg, wu)
    assert all(not t.any() for t in zero)


@pytest.mark.parametrize("t", [3, 40])
def test_what_is_kept_over_its_range(t):
    """Gates and ups from 2^-45 to 2^44 (and 2^120, and NaN): one input channel and weights of every size."""
    x = torch.zeros(t, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    x[1, 0] = -1.0
    w = torch.zeros(256, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = (1.0 + torch.rand(256, generator=torch.Generator().manual_seed(3))).cuda() * torch.exp2(torch.arange(256, device="cuda") % 90 - 45.0)
    w[8, 0], w[9, 0] = float("nan"), 2.0 ** 120
    _, ka, kb = mpg.gated_gemm(x, w, w, keep=True)
    ok()
    g = x[:, :1].double() @ w[:, :1].double().t()
    a, d = plain.act(g, "silu")
    for k, exact in ((ka, a), (kb, g * d)):
        v = plain.kept_values(k)
        inside = (exact.abs() < 2.0 ** 32) & ~exact.isnan()
        off = (v - exact).abs()
        # (far below 0 act and act' vanish; what is left of them is off by the exponential's argument)
        assert bool((off[inside] <= ((2.0 ** -10 + plain.ACT) * exact.abs() + 2.0 ** -40)[inside]).all())
        assert v[:, 8].isnan().all() and v[0, 9].isinf() and bool((v[0][exact[0].abs() >= 2.0 ** 33].isinf()).all())


@pytest.mark.parametrize("t", [5, 100])
def test_without_elements(t):
    dev = "cuda"
    e = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    assert mpg.gated_gemm(e(0, 8), e(6, 8), e(6, 8)).shape == (0, 6)
    assert mpg.gated_gemm(e(t, 8), e(0, 8), e(0, 8)).shape == (t, 0)
    y, g, u = mpg.gated_gemm(e(t, 0), e(6, 0), e(6, 0), keep=True)
    assert y.shape == (t, 6) and not y.any() and not g.any() and not u.any()
    dx, dwg, dwu = mpg.gated_gemm_backward(e(0, 6), e(0, 8), e(6, 8), e(6, 8))
    assert dx.shape == (0, 8) and not dwg.any() and not dwu.any()
    dx, dwg, dwu = mpg.gated_gemm_backward(e(t, 0), e(t, 8), e(0, 8), e(0, 8))
    assert dx.shape == (t, 8) and not dx.any() and dwg.shape == (0, 8)
    assert mpg.gated_gemm_backward(e(t, 6), e(t, 0), e(6, 0), e(6, 0))[0].shape == (t, 0)
    ok()


@pytest.mark.parametrize("t", [4, 40, 600])
def test_a_token_that_is_no_number_stays_alone(t):
    x, wg, wu, dy = operands(t, 64, 96, "bf16", 8)
    good = mpg.gated_gemm(x, wg, wu)
    gx = mpg.gated_gemm_backward(dy, x, wg, wu)[0]
    x[t // 2, 5] = float("nan")
    y = mpg.gated_gemm(x, wg, wu)
    dx, dwg, _ = mpg.gated_gemm_backward(dy, x, wg, wu)
    ok()
    others = torch.arange(t, device="cuda") != t // 2
    assert y[t // 2].isnan().all() and torch.equal(y[others], good[others])
    assert dx[t // 2].isnan().all() and torch.equal(dx[others], gx[others]) and dwg.isnan().all()


@pytest.mark.parametrize("t", [3, 20, 50, 300])
def test_nothing_is_written_beyond_the_results(t):
    h, i, pad = 72, 100, 5
    x, wg, wu, dy = operands(t, h, i, "bf16", 9)
    mark = 12345.0
    lay = mpg.GatedLayer(t, h, i, mpg.BF16, 0, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), h, h, h)

    def room(rows, cols):
        return torch.full((rows + 2, cols + pad), mark, dtype=torch.bfloat16, device="cuda")
    import ctypes
    y, g, u = room(t, i), room(t, i).view(torch.int16), room(t, i).view(torch.int16)
    gap = int(g[-1, -1])
    need = int(mpg.lib().mpg_gated_gemm_workspace_size(ctypes.byref(lay)))
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    mpg.gated_gemm_raw(lay, *(v for b in (y, g, u) for v in (b.data_ptr(), i + pad)), ws.data_ptr(), need)
    ok()
    assert (ws[need:] == 77).all()
    need = int(mpg.lib().mpg_gated_gemm_backward_workspace_size(ctypes.byref(lay)))
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    outs = [room(t, h), room(i, h), room(i, h)]
    mpg.gated_gemm_backward_raw(lay, dy.data_ptr(), i, g.data_ptr(), i + pad, u.data_ptr(), i + pad,
                                *(v for b in outs for v in (b.data_ptr(), h + pad)), ws.data_ptr(), need)
    ok()
    assert (ws[need:] == 77).all()
    for b, rows, cols in ((y, t, i), (g, t, i), (u, t, i), (outs[0], t, h), (outs[1], i, h), (outs[2], i, h)):
        m = gap if b.dtype == torch.int16 else mark
        assert (b[rows:] == m).all() and (b[:, cols:] == m).all() and not (b[:rows, :cols] == m).all(dim=1).any()
    # lines with gaps give the same values
    ref = mpg.gated_gemm_backward(dy, x, wg, wu, kept=(g[:t, :i], u[:t, :i]))
    for b, r in zip(outs, ref):
        assert torch.equal(b[:r.shape[0], :r.shape[1]], r)


@pytest.mark.parametrize("t", [20, 70, 1060])
def test_large_packed_results_of_odd_lines(t):
    """Results of a million elements whose lines are off 16 bytes, with marks before and behind them."""
    import ctypes
    h, i = 1001, 1060
    x, wg, wu, dy = operands(t, h, i, "bf16", 13)
    lay = mpg.GatedLayer(t, h, i, mpg.BF16, 0, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), h, h, h)
    mark = 12352.0
    outs = [torch.full((16 + r * h + 16,), mark, dtype=torch.bfloat16, device="cuda") for r in (t, i, i)]
    need = int(mpg.lib().mpg_gated_gemm_backward_workspace_size(ctypes.byref(lay)))
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    refs, bounds = plain.gated_gradients(dy, x, wg, wu, "silu")
    for shift in (16, 8, 9):                          # (9: not on 16 bytes, written as it comes)
        for b in outs:
            b.fill_(mark)
        mpg.gated_gemm_backward_raw(lay, dy.data_ptr(), i, 0, 0, 0, 0, *(v for b in outs for v in (b[shift:].data_ptr(), h)),
                                    ws.data_ptr(), need)
        ok()
        assert (ws[need:] == 77).all()
        for b, r, e in zip(outs, refs, bounds):
            n = r.numel()
            plain.check(b[shift:shift + n].view(r.shape), r, e)
            assert (b[:shift] == mark).all() and (b[shift + n:] == mark).all()


@pytest.mark.parametrize("t", [1, 5, 16, 30, 60, 64, 65])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_lines_of_odd_length_on_aligned_places(t, dtype):
    """100 columns (and 77 inner values) in lines of 104 and 80 elements, all on 16 bytes: chunks cut by the
    matrix's edge, the last line's end at the end of its memory, and gaps that stay as they were."""
    import ctypes
    h, i, ldh, ldi = 100, 77, 104, 80
    code = mpg.BF16 if dtype == "bf16" else mpg.F16

    def lined(m, ld):
        flat = torch.full(((m.shape[0] - 1) * ld + m.shape[1],), float("nan"), dtype=m.dtype, device="cuda")
        v = flat.as_strided(m.shape, (ld, 1))
        v.copy_(m)
        return v
    x, wg, wu, dy = operands(t, h, i, dtype, 12)
    x, wg, wu, dy = lined(x, ldh), lined(wg, ldh), lined(wu, ldh), lined(dy, ldi)
    lay = mpg.GatedLayer(t, h, i, code, 0, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), ldh, ldh, ldh)
    mark = 12345.0 if dtype == "fp16" else 12352.0
    outs = [torch.full((r + 1, ldh), mark, dtype=x.dtype, device="cuda") for r in (t, i, i)]
    y = torch.full((t + 1, ldi), mark, dtype=x.dtype, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    need = int(mpg.lib().mpg_gated_gemm_backward_workspace_size(ctypes.byref(lay)))
    assert need <= ws.numel()
    mpg.gated_gemm_raw(lay, y.data_ptr(), ldi, 0, 0, 0, 0, ws.data_ptr(), ws.numel())
    mpg.gated_gemm_backward_raw(lay, dy.data_ptr(), ldi, 0, 0, 0, 0, *(v for b in outs for v in (b.data_ptr(), ldh)),
                                ws.data_ptr(), ws.numel())
    ok()
    (ref, _, _), (bound, _, _) = plain.gated(x, wg, wu, "silu")
    plain.check(y[:t, :i], ref, bound)
    refs, bounds = plain.gated_gradients(dy, x, wg, wu, "silu")
    for o, r, b in zip(outs, refs, bounds):
        plain.check(o[:-1, :h], r, b)
        assert (o[-1] == mark).all() and (o[:, h:] == mark).all()
    assert (y[-1] == mark).all() and (y[:, i:] == mark).all()


def test_a_given_workspace_streams_threads_and_graphs():
    x, wg, wu, dy = operands(200, 136, 264, "fp16", 10)
    y, g, u = mpg.gated_gemm(x, wg, wu, keep=True)
    ref = mpg.gated_gemm_backward(dy, x, wg, wu, kept=(g, u))
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    for a, b in zip(ref, mpg.gated_gemm_backward(dy, x, wg, wu, kept=(g, u), workspace=ws)):
        assert torch.equal(a, b)
    with pytest.raises(Exception):
        mpg.gated_gemm_backward(dy, x, wg, wu, workspace=ws[:16])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(mpg.gated_gemm(x, wg, wu, stream=side), y)
    side.synchronize()
    # two threads, a stream each
    results = [None, None]

    def work(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            results[k] = [mpg.gated_gemm_backward(dy, x, wg, wu, kept=(g, u)) for _ in range(20)]
        s.synchronize()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for r in results:
        for outs in r:
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    # captured, replayed with other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cy, cg, cu = mpg.gated_gemm(x, wg, wu, keep=True)
        couts = mpg.gated_gemm_backward(dy, x, wg, wu, kept=(cg, cu))
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    y2, g2, u2 = mpg.gated_gemm(x, wg, wu, keep=True)
    ref2 = mpg.gated_gemm_backward(dy, x, wg, wu, kept=(g2, u2))
    assert torch.equal(cy, y2) and all(torch.equal(a, b) for a, b in zip(couts, ref2)) and not torch.equal(cy, y)
    ok()


def test_calls_that_the_plain_path_leaves_to_python():
    """The Python form and the extension make the same calls."""
    x, wg, wu, dy = operands(40, 64, 96, "bf16", 11)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    assert torch.equal(mpg.gated_gemm(x, wg, wu, workspace=ws), mpg.gated_gemm(x, wg, wu))
    for bad in (lambda: mpg.gated_gemm(x, wg, wu[:-1]), lambda: mpg.gated_gemm(x, wg[:, :-8], wu[:, :-8]),
                lambda: mpg.gated_gemm(x[0], wg, wu), lambda: mpg.gated_gemm(x.t().contiguous().t(), wg, wu),
                lambda: mpg.gated_gemm_backward(dy[:-1], x, wg, wu),
                lambda: mpg.gated_gemm_backward(dy, x, wg, wu, kept=(dy.view(torch.int16), None)),
                lambda: mpg.gated_gemm_backward(dy, x, wg, wu, kept=(dy.view(torch.int16), dy.view(torch.int16)[:, 1:])),
                lambda: mpg.gated_gemm(x, wg.cpu(), wu)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mpg.gated_gemm(x.float(), wg.float(), wu.float()), lambda: mpg.gated_gemm(x, wg.half(), wu),
                lambda: mpg.gated_gemm_backward(dy, x, wg, wu, kept=(dy, dy))):
        with pytest.raises(TypeError):
            bad()
    one = x[:1].expand(40, 64)
    with pytest.raises(ValueError):
        mpg.gated_gemm(one, wg, wu)
