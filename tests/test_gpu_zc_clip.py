"""GPU: the norm of many gradients and their clipping against 64 bits."""
import pytest

import mixed_precision_matmul_gb300 as mpg

torch = pytest.importorskip("torch")
import fused_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def ok():
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK


def norm_of(grads):
    return float(sum((g.double() ** 2).sum() for g in grads) ** 0.5)


def check(grads, max_norm, out=None, eps=1e-6):
    """Runs a call and holds its results to 64 bits.  The norm: eight squares in fp32 (each
    of eight additions 2^-24 at most), then 64 bits, halved by the root, rounded once.  The
    factor: that, an addition, a division and a product, 2^-24 each."""
    before = [g.clone() for g in grads]
    ref = norm_of(before)
    norm = mpg.clip_grad_norm(grads, max_norm, out=out, eps=eps)
    ok()
    assert norm.shape == () and norm.dtype == F32
    assert abs(float(norm) - ref) <= 6 * 2.0 ** -24 * ref
    f = min(1.0, max_norm / (ref + eps))
    for b, o in zip(before, grads if out is None else out):
        r = b.double() * f
        plain.check(o, r, 10 * 2.0 ** -24 * r.abs())
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(before, grads))
    return norm


SIZES = [0, 1, 7, 8, 9, 255, 2047, 2048, 2049, 8191, 8192, 8193, 100000]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_sizes_and_types(dtype):
    g = torch.Generator("cuda").manual_seed(1)
    grads = [torch.randn(n, device="cuda", generator=g).to(dtype) for n in SIZES]
    for out_type in (F32, F16, BF16):
        check(grads, 1.0, [torch.empty(n, dtype=out_type, device="cuda") for n in SIZES])
    check(grads, 1e9, [torch.empty_like(t) for t in grads])
    check(grads, 2.5)
    check([grads[1]], 0.5)
    check([grads[0], grads[2]], 0.0)


@pytest.mark.parametrize("most", [262144 - 2048, 262144, 262145, 700001])
def test_around_what_one_launch_holds(most):
    g = torch.Generator("cuda").manual_seed(8)
    for dtype in (F32, BF16):
        grads = [torch.randn(n, device="cuda", generator=g).to(dtype) for n in (most - 5000, 2999, 2001)]
        check(grads, 1.0, [torch.empty_like(t, dtype=F32) for t in grads])
        check(grads, 1e9)
        check(grads, 0.25)


def test_mixed_types_shapes_and_alignment():
    g = torch.Generator("cuda").manual_seed(2)
    flat = torch.randn(300000, device="cuda", generator=g)
    grads = [flat[1:30001], flat[30001:60001].view(300, 100).t(), flat[60004:90004].to(F16)[3:], flat[90004:180004].to(BF16).view(90, 10, 100),
             torch.randn((), device="cuda", generator=g), flat[200000:200001]]
    check(grads, 1.0, [torch.empty_like(t) for t in grads])
    check(grads, 1.0, [torch.empty_like(t, dtype=F32) for t in grads])
    check(grads, 1.0)


@pytest.mark.parametrize("count", [63, 64, 65, 897, 2000])
def test_many_tensors(count):
    g = torch.Generator("cuda").manual_seed(3)
    flat = torch.randn(count * 40, device="cuda", generator=g)
    grads = [flat[40 * i:40 * i + i % 41] for i in range(count)]
    check(grads, 1.0, [torch.empty_like(t) for t in grads])
    check(grads, 3.0)


def test_a_large_set():
    g = torch.Generator("cuda").manual_seed(4)
    grads = [torch.randn(5_000_001, device="cuda", generator=g).to(BF16), torch.randn(30_000_000, device="cuda", generator=g)]
    check(grads, 1.0, [torch.empty_like(t) for t in grads])
    a = [torch.empty_like(t) for t in grads]
    b = [torch.empty_like(t) for t in grads]
    assert torch.equal(mpg.clip_grad_norm(grads, 1.0, out=a), mpg.clip_grad_norm(grads, 1.0, out=b))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e18, 1e30, 1e34])
def test_squares_that_fp32_cannot_hold(scale):
    g = torch.Generator("cuda").manual_seed(5)
    for dtype in (F32, BF16):
        grads = [(scale * torch.randn(n, device="cuda", generator=g, dtype=torch.float64)).to(dtype) for n in (50000, 3)]
        ref = norm_of(grads)
        out = [torch.empty_like(t) for t in grads]
        norm = mpg.clip_grad_norm(grads, ref / 2, out=out, eps=0.0)
        ok()
        assert abs(float(norm) - ref) <= 6 * 2.0 ** -24 * ref + 2.0 ** -149
        for t, o in zip(grads, out):
            r = t.double() / 2
            plain.check(o, r, 1e-6 * r.abs() + (2.0 ** -148 if scale < 1e-30 else 0.0))


def test_large_beside_small():
    """Squares of one tensor overflow fp32, the other's underflow it."""
    grads = [torch.full((1000,), 1e25, device="cuda"), torch.full((1000,), 1e-30, device="cuda")]
    check(grads, 1.0, [torch.empty_like(t) for t in grads])


def test_zeros():
    grads = [torch.zeros(20000, device="cuda"), torch.zeros(5, dtype=F16, device="cuda")]
    assert float(mpg.clip_grad_norm(grads, 1.0)) == 0.0
    assert float(mpg.clip_grad_norm(grads, 0.0)) == 0.0
    assert float(mpg.clip_grad_norm([torch.zeros(0, device="cuda")], 1.0)) == 0.0
    assert not any(t.any() for t in grads)
    # 0 / 0: max_norm 0 without eps
    mpg.clip_grad_norm(grads, 0.0, eps=0.0)
    assert grads[0].isnan().all()


def test_gradients_that_are_no_numbers():
    def fresh():
        return [torch.ones(3000, device="cuda"), torch.ones(50, dtype=BF16, device="cuda")]
    a = fresh()
    a[0][1234] = float("nan")
    assert mpg.clip_grad_norm(a, 1.0).isnan()
    assert all(t.isnan().all() for t in a)
    a = fresh()
    a[1][7] = -float("inf")
    assert float(mpg.clip_grad_norm(a, 1.0)) == float("inf")
    assert a[1][7].isnan() and not a[0].any() and int((a[1] != 0).sum()) == 1
    a = fresh()
    a[1][7] = float("inf")
    assert float(mpg.clip_grad_norm(a, float("inf"))) == float("inf")
    assert int((a[1] == 1).sum()) == 49 and bool((a[0] == 1).all())
    a = fresh()
    before = [t.clone() for t in a]
    n = mpg.clip_grad_norm(a, float("inf"))
    assert abs(float(n) - 3050 ** 0.5) < 1e-4 and all(torch.equal(x, y) for x, y in zip(a, before))
    ok()


def test_refusals_of_the_torch_form():
    a, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    for bad in (lambda: mpg.clip_grad_norm([a, a], 1.0), lambda: mpg.clip_grad_norm([a, b], 1.0, out=[b, a]),
                lambda: mpg.clip_grad_norm([a], 1.0, out=[b[1:]]), lambda: mpg.clip_grad_norm([a.view(8, 8)[:, ::2]], 1.0),
                lambda: mpg.clip_grad_norm([a[:1].expand(8)], 1.0), lambda: mpg.clip_grad_norm([a], -1.0),
                lambda: mpg.clip_grad_norm([a.view(8, 8)], 1.0, out=[b.view(8, 8).t()]), lambda: mpg.clip_grad_norm([a, b.cpu()], 1.0)):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    with pytest.raises(TypeError):
        mpg.clip_grad_norm([a.double()], 1.0)
    assert torch.equal(a, torch.ones_like(a)) and torch.equal(b, torch.ones_like(b))
    check([a, a], 1.0, [torch.empty_like(a), torch.empty_like(a)])      # read twice: counted twice


def test_graph_stream_and_workspace():
    g = torch.Generator("cuda").manual_seed(6)
    grads = [torch.randn(n, device="cuda", generator=g) for n in (1000, 70000)]
    out = [torch.empty_like(t) for t in grads]
    norm = mpg.clip_grad_norm(grads, 1.0, out=out)
    graph = torch.cuda.CUDAGraph()
    out2 = [torch.empty_like(t) for t in grads]
    with torch.cuda.graph(graph):
        n2 = mpg.clip_grad_norm(grads, 1.0, out=out2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(out, out2))
    grads[0].mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n2, mpg.clip_grad_norm(grads, 1.0, out=out)) and all(torch.equal(a, b) for a, b in zip(out, out2))
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(mpg.clip_grad_norm(grads, 1.0, out=out2, workspace=ws, stream=side), n2)
    assert torch.equal(mpg.clip_grad_norm(iter(grads), 1.0, out=iter(out2), stream=side), n2)
    side.synchronize()
    with pytest.raises(Exception):
        mpg.clip_grad_norm(grads, 1.0, out=out2, workspace=ws[:8])
    ok()
