"""GPU: the cross entropy of a projection and its gradients against 64 bits."""
import pytest

import mixed_precision_matmul_gb300 as mpg

torch = pytest.importorskip("torch")
import fused_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def operands(t, h, v, dtype, seed=0, pad=0, shift=0, ignored=0.3, scale=2.0):
    g = torch.Generator().manual_seed(seed)

    def make(rows, cols, s):
        buf = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=TYPES[dtype], device="cuda")
        m = buf[shift:].view(rows, cols + pad)[:, :cols]
        m.copy_((s * torch.randn(rows, cols, generator=g)).to(TYPES[dtype]))
        return m
    x, w = make(t, h, 1.0), make(v, h, scale * h ** -0.5)
    target = torch.randint(0, v, (t,), generator=g)
    target[torch.rand(t, generator=g) < ignored] = -100
    return x, w, target.cuda()


def ok():
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK


SHAPES = [(1, 1, 1), (1, 64, 1000), (3, 100, 33), (8, 513, 40), (9, 64, 1003), (16, 1000, 15), (17, 72, 129), (32, 520, 5003),
          (33, 64, 64), (33, 1, 5), (40, 72, 1), (64, 100, 1003), (127, 128, 65), (130, 65, 70), (257, 200, 129), (300, 1001, 515)]


@pytest.mark.parametrize("t,h,v", SHAPES + [(2048, 264, 4099), (600, 512, 20000), (200, 4000, 300), (40, 3999, 70), (600, 4096, 1003)])
def test_loss(t, h, v):
    for dtype, pad, shift in (("bf16", 0, 0), ("fp16", 8, 8), ("bf16", 3, 1)):
        x, w, target = operands(t, h, v, dtype, 1, pad, shift)
        (value, lse), (ev, el) = plain.loss(x, w, target)
        for tg in (target, target.int(), torch.stack([target, target], 1)[:, 1]):
            a, b = mpg.linear_cross_entropy(x, w, tg)
            ok()
            plain.check(a, value, ev)
            plain.check(b, lse, el)


@pytest.mark.parametrize("t,h,v", SHAPES + [(2000, 264, 4099), (40, 64, 30000), (5, 72, 50000), (200, 4000, 300), (40, 3999, 70), (600, 4096, 1003),
                                             (9, 1001, 1100), (40, 1003, 1100), (300, 1001, 1100), (1100, 1001, 130)])
def test_gradients(t, h, v):
    for dtype, pad, shift in (("fp16", 0, 0), ("bf16", 8, 8), ("fp16", 3, 1)):
        x, w, target = operands(t, h, v, dtype, 2, pad, shift)
        _, lse = mpg.linear_cross_entropy(x, w, target)
        weights = torch.rand(t, generator=torch.Generator().manual_seed(5)).cuda() + 0.1
        for dloss in ((256.0 / torch.tensor(float(t))).cuda().expand(t), weights, torch.stack([weights, weights], 1)[:, 0]):
            refs, bounds = plain.loss_gradients(x, w, target, lse, dloss)
            outs = mpg.linear_cross_entropy_backward(x, w, target, lse, dloss)
            ok()
            for o, r, b in zip(outs, refs, bounds):
                plain.check(o, r, b)


def test_pieces_of_the_vocabulary():
    """8192 tokens and 40000 classes: the logits' gradient (655 MB) in two pieces."""
    t, h, v = 8192, 72, 40000
    x, w, target = operands(t, h, v, "bf16", 3)
    value, lse = mpg.linear_cross_entropy(x, w, target)
    dloss = torch.ones((), device="cuda").expand(t)
    dx, dw = mpg.linear_cross_entropy_backward(x, w, target, lse, dloss)
    ok()
    rows = torch.arange(0, t, 61, device="cuda")
    (rv, rl), (ev, el) = plain.loss(x[rows], w, target[rows])
    plain.check(value[rows], rv, ev)
    plain.check(lse[rows], rl, el)
    (rx, _), (ex, _) = plain.loss_gradients(x[rows], w, target[rows], lse[rows], dloss[rows])
    plain.check(dx[rows], rx, ex)
    # dW of some classes, by the whole of x
    cols = torch.cat([torch.arange(0, v, 997, device="cuda"), torch.tensor([19967, 19968, 20223, 20224, v - 1], device="cuda")])
    l = x.double() @ w[cols].double().t()
    p = torch.exp(l - lse.double()[:, None])
    d = (p - (target[:, None] == cols[None]).double()) * (target != -100)[:, None]
    el = plain.sum_error(h) * (x.double().abs() @ w[cols].double().abs().t()) + 2 * 2.0 ** -23 * (l.abs() + lse.double().abs()[:, None]) + 2.0 ** -22
    ed = (target != -100)[:, None] * (p * torch.expm1(el) + plain.half_step(torch.bfloat16) * d.abs())
    plain.check(dw[cols], d.t() @ x.double(), ed.t() @ x.double().abs() + plain.sum_error(t) * (d.abs().t() @ x.double().abs()))


def test_gradient_against_differences():
    x, w, target = operands(50, 72, 300, "bf16", 4)
    _, lse = mpg.linear_cross_entropy(x, w, target)
    dloss = torch.rand(50, generator=torch.Generator().manual_seed(1)).cuda()
    outs = mpg.linear_cross_entropy_backward(x, w, target, lse, dloss)
    ok()
    refs, bounds = plain.loss_gradients(x, w, target, lse, dloss)
    base = [x.double(), w.double()]
    for k in range(2):
        d = torch.randn(base[k].shape, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
        s = 1e-5

        def f(step):
            a = [t + step * d if j == k else t for j, t in enumerate(base)]
            l = a[0] @ a[1].t()
            v = torch.logsumexp(l, 1) - l.gather(1, target.clamp(min=0)[:, None])[:, 0]
            return float((torch.where(target == -100, 0.0, v) * dloss).sum())
        slope = (f(s) - f(-s)) / (2 * s)
        allowed = float(((bounds[k] + plain.half_step(torch.bfloat16) * refs[k].abs()) * d.abs()).sum()) + 1e-6
        # (the gradient is taken at the kernel's lse, 2^-18 off at most)
        allowed += 2.0 ** -18 * float((refs[k].abs() * d.abs()).sum())
        assert abs(float((outs[k].double() * d).sum()) - slope) <= allowed


@pytest.mark.parametrize("t", [4, 70])
def test_every_token_ignored(t):
    x, w, target = operands(t, 64, 500, "fp16", 5, ignored=2.0)
    value, lse = mpg.linear_cross_entropy(x, w, target)
    assert not value.any() and not lse.any()
    # the mean over no tokens: its gradient is infinite, and not used
    for bad in (float("inf"), float("nan")):
        dx, dw = mpg.linear_cross_entropy_backward(x, w, target, lse, torch.full((t,), bad, device="cuda"))
        assert not dx.any() and not dw.any()
    ok()


@pytest.mark.parametrize("t", [6, 70])
def test_an_ignored_class(t):
    """ignore_index may be a class; -100 is then none."""
    x, w, target = operands(t, 64, 500, "bf16", 6, ignored=0.0)
    target[::3] = 7
    value, lse = mpg.linear_cross_entropy(x, w, target, ignore_index=7)
    (rv, rl), (ev, el) = plain.loss(x, w, target, 7)
    plain.check(value, rv, ev)
    plain.check(lse, rl, el)
    dloss = torch.ones(t, device="cuda")
    refs, bounds = plain.loss_gradients(x, w, target, lse, dloss, 7)
    for o, r, b in zip(mpg.linear_cross_entropy_backward(x, w, target, lse, dloss, ignore_index=7), refs, bounds):
        plain.check(o, r, b)


@pytest.mark.parametrize("t", [6, 70])
def test_a_target_that_is_no_class(t):
    x, w, target = operands(t, 64, 500, "bf16", 7, ignored=0.2)
    good = mpg.linear_cross_entropy(x, w, target)
    for bad in (500, -1, 2 ** 40, -2 ** 62):
        wrong = target.clone()
        wrong[2] = bad
        value, lse = mpg.linear_cross_entropy(x, w, wrong)
        others = torch.arange(t, device="cuda") != 2
        assert value[2].isnan() and lse[2].isnan() and torch.equal(value[others], good[0][others])
        dx, dw = mpg.linear_cross_entropy_backward(x, w, wrong, lse, torch.ones(t, device="cuda"))
        assert dx[2].isnan().all() and not dx[others].isnan().any() and dw.isnan().all()
    ok()


@pytest.mark.parametrize("t", [6, 70])
def test_large_logits_and_no_numbers(t):
    x, w, target = operands(t, 64, 500, "bf16", 8, ignored=0.0)
    x *= 1000.0                                       # logits of thousands: no exponential overflows
    value, lse = mpg.linear_cross_entropy(x, w, target)
    (rv, rl), (ev, el) = plain.loss(x, w, target)
    plain.check(value, rv, ev)
    plain.check(lse, rl, el)
    dloss = torch.ones(t, device="cuda")
    dx, dw = mpg.linear_cross_entropy_backward(x, w, target, lse, dloss)
    assert not dx.isnan().any() and not dw.isnan().any()
    # a NaN stays in its row; logits of +infinity make an infinite lse, of -infinity count nothing
    x, w, target = operands(t, 64, 500, "bf16", 9, ignored=0.0)
    x[1, 3] = float("nan")
    value, lse = mpg.linear_cross_entropy(x, w, target)
    assert value[1].isnan() and lse[1].isnan() and not value[torch.arange(t, device="cuda") != 1].isnan().any()
    x[1] = 0.0
    x[1, 0] = 1.0
    x[2] = x[1]
    w[:, 0] = 0.0
    w[3, 0] = float("inf")
    w[4, 0] = -float("inf")
    x[3:, 0] = 0.0
    x[0, 0] = 0.0
    target[:] = 7
    value, lse = mpg.linear_cross_entropy(x[1:3], w, target[1:3])
    assert (lse == float("inf")).all()
    w[3, 0] = -float("inf")
    value, lse = mpg.linear_cross_entropy(x[1:3], w, target[1:3])
    expected = torch.log(torch.tensor(498.0, dtype=torch.float64)).expand(2).cuda()
    plain.check(value, expected, torch.full_like(expected, 2.0 ** -19))
    w[:, 0] = -float("inf")
    value, lse = mpg.linear_cross_entropy(x[1:3], w, target[1:3])
    assert (lse == -float("inf")).all()
    ok()


def test_small_probabilities_in_fp16():
    """One class of 40000 has most of the mass: the others' gradients (2^-16 .. 2^-27 of dloss,
    itself 2^-13) are below fp16's normal numbers and come out all the same."""
    t, h, v = 64, 64, 40000
    x, w, target = operands(t, h, v, "fp16", 10, ignored=0.0, scale=0.01)
    _, lse = mpg.linear_cross_entropy(x, w, target)
    dloss = torch.full((t,), 2.0 ** -4, device="cuda")
    refs, bounds = plain.loss_gradients(x, w, target, lse, dloss)
    outs = mpg.linear_cross_entropy_backward(x, w, target, lse, dloss)
    ok()
    for o, r, b in zip(outs, refs, bounds):
        plain.check(o, r, b)


def test_what_is_not_needed_and_without_tokens():
    x, w, target = operands(70, 64, 300, "bf16", 11)
    _, lse = mpg.linear_cross_entropy(x, w, target)
    d = torch.ones(70, device="cuda")
    full = mpg.linear_cross_entropy_backward(x, w, target, lse, d)
    dx, none = mpg.linear_cross_entropy_backward(x, w, target, lse, d, need_dw=False)
    assert none is None and torch.equal(dx, full[0])
    none, dw = mpg.linear_cross_entropy_backward(x, w, target, lse, d, need_dx=False)
    assert none is None and torch.equal(dw, full[1])
    value, lse = mpg.linear_cross_entropy(x[:0], w, target[:0])
    assert value.shape == (0,) and lse.shape == (0,)
    dx, dw = mpg.linear_cross_entropy_backward(x[:0], w, target[:0], lse, d[:0])
    assert dx.shape == (0, 64) and dw.shape == (300, 64) and not dw.any()
    ok()


@pytest.mark.parametrize("t", [5, 300])
def test_nothing_is_written_beyond_the_results(t):
    import ctypes
    h, v, pad = 72, 203, 5
    x, w, target = operands(t, h, v, "bf16", 12)
    d = mpg.VocabLoss(t, h, v, mpg.BF16, x.data_ptr(), w.data_ptr(), h, h, target.data_ptr(), 8, 1, -100)
    loss, lse = (torch.full((t + 3,), 9.0, device="cuda") for _ in range(2))
    need = int(mpg.lib().mpg_linear_cross_entropy_workspace_size(ctypes.byref(d)))
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    mpg.linear_cross_entropy_raw(d, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), need)
    ok()
    assert (ws[need:] == 77).all() and (loss[t:] == 9.0).all() and (lse[t:] == 9.0).all()
    need = int(mpg.lib().mpg_linear_cross_entropy_backward_workspace_size(ctypes.byref(d)))
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    dx, dw = (torch.full((r + 2, h + pad), 12345.0, dtype=torch.bfloat16, device="cuda") for r in (t, v))
    mpg.linear_cross_entropy_backward_raw(d, lse.data_ptr(), one.data_ptr(), 0, dx.data_ptr(), h + pad, dw.data_ptr(), h + pad,
                                          ws.data_ptr(), need)
    ok()
    assert (ws[need:] == 77).all()
    for b, rows in ((dx, t), (dw, v)):
        assert (b[rows:] == 12345.0).all() and (b[:, h:] == 12345.0).all() and not (b[:rows, :h] == 12345.0).any()
    ref = mpg.linear_cross_entropy_backward(x, w, target, lse[:t], one.expand(t))
    assert torch.equal(dx[:t, :h], ref[0]) and torch.equal(dw[:v, :h], ref[1])


@pytest.mark.parametrize("t", [1, 5, 16, 30, 60, 64, 65])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_lines_of_odd_length_on_aligned_places(t, dtype):
    """100 columns in lines of 104 elements, all on 16 bytes, the last line's end at the end of its memory."""
    h, v, ld = 100, 203, 104

    def lined(m):
        flat = torch.full(((m.shape[0] - 1) * ld + h,), float("nan"), dtype=m.dtype, device="cuda")
        r = flat.as_strided(m.shape, (ld, 1))
        r.copy_(m)
        return r
    x, w, target = operands(t, h, v, dtype, 14, ignored=0.2)
    x, w = lined(x), lined(w)
    value, lse = mpg.linear_cross_entropy(x, w, target)
    (rv, rl), (ev, el) = plain.loss(x, w, target)
    plain.check(value, rv, ev)
    plain.check(lse, rl, el)
    d = mpg.VocabLoss(t, h, v, mpg.BF16 if dtype == "bf16" else mpg.F16, x.data_ptr(), w.data_ptr(), ld, ld, target.data_ptr(), 8, 1, -100)
    dloss = torch.rand(t, generator=torch.Generator().manual_seed(2)).cuda() + 0.1
    mark = 12345.0 if dtype == "fp16" else 12352.0
    outs = [torch.full((r + 1, ld), mark, dtype=x.dtype, device="cuda") for r in (t, v)]
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    mpg.linear_cross_entropy_backward_raw(d, lse.data_ptr(), dloss.data_ptr(), 1, outs[0].data_ptr(), ld, outs[1].data_ptr(), ld,
                                          ws.data_ptr(), ws.numel())
    ok()
    refs, bounds = plain.loss_gradients(x, w, target, lse, dloss)
    for o, r, b in zip(outs, refs, bounds):
        plain.check(o[:-1, :h], r, b)
        assert (o[-1] == mark).all() and (o[:, h:] == mark).all()


def test_graph_stream_and_python_form():
    x, w, target = operands(100, 136, 1003, "fp16", 13)
    d = torch.full((), 0.01, device="cuda").expand(100)
    value, lse = mpg.linear_cross_entropy(x, w, target)
    ref = mpg.linear_cross_entropy_backward(x, w, target, lse, d)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    assert torch.equal(mpg.linear_cross_entropy(x, w, target, workspace=ws)[0], value)
    for a, b in zip(ref, mpg.linear_cross_entropy_backward(x, w, target, lse, d, workspace=ws)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(mpg.linear_cross_entropy(x, w, target, stream=side)[1], lse)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cv, cl = mpg.linear_cross_entropy(x, w, target)
        cg = mpg.linear_cross_entropy_backward(x, w, target, cl, d)
    x.mul_(0.5)
    target.copy_(target.roll(1))
    graph.replay()
    torch.cuda.synchronize()
    v2, l2 = mpg.linear_cross_entropy(x, w, target)
    assert torch.equal(cv, v2) and torch.equal(cl, l2) and not torch.equal(cv, value)
    assert all(torch.equal(a, b) for a, b in zip(cg, mpg.linear_cross_entropy_backward(x, w, target, l2, d)))
    for bad in (lambda: mpg.linear_cross_entropy(x, w[:, :8], target), lambda: mpg.linear_cross_entropy(x, w, target[1:]),
                lambda: mpg.linear_cross_entropy(x, w, target.cpu()), lambda: mpg.linear_cross_entropy(x, w, target[:, None]),
                lambda: mpg.linear_cross_entropy_backward(x, w, target, lse[1:], d),
                lambda: mpg.linear_cross_entropy_backward(x, w, target, lse[:1].expand(100), d)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mpg.linear_cross_entropy(x.float(), w.float(), target), lambda: mpg.linear_cross_entropy(x, w, target.half()),
                lambda: mpg.linear_cross_entropy_backward(x, w, target, lse, d.half())):
        with pytest.raises(TypeError):
            bad()
    ok()
