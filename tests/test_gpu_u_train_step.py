"""GPU: the 8-bit products and the orthogonalised update together, as the
example trains with them: the losses are the exact training's, the gradients are those of the exact
layer within what 8-bit operands allow, and a step replays from a graph."""
import importlib.util
import os

import pytest

import mixed_precision_matmul_gb300 as mpg

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    mpg.build()
    spec = importlib.util.spec_from_file_location("fp8_muon_step", os.path.join(ROOT, "examples", "fp8_muon_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_losses(tokens, inputs, outputs, steps, rate, mu, decay, seed):
    """The example's training on the same draws in 64 bits: nothing is rounded to 8."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(*shape):
        return torch.randn(shape, generator=g, device="cuda").double()
    teacher = draw(outputs, inputs) / inputs ** 0.5
    w = torch.zeros_like(teacher)
    momentum = torch.zeros_like(teacher)
    a, b, c = mpg.NS_COEFFS
    losses = []
    for _ in range(steps):
        x = draw(tokens, inputs)
        diff = x @ (w - teacher).t()
        losses.append(float(diff.square().mean()))
        momentum = mu * momentum + (diff * (2.0 / diff.numel())).t() @ x
        o = momentum / momentum.norm()
        for _ in range(5):
            q = o @ o.t()
            o = a * o + (b * q + c * q @ q) @ o
        w = (1 - rate * decay) * w - rate * o
    return losses


def test_losses_are_the_exact_training_s(example):
    """Step by step against 64 bits.  Half a step of e4m3 is 2^-4 of the value, so
    the outputs' errors add at most 2 * 2^-8 of their mean square (at most 1) to a
    loss.  The gradient's operands are off by at most 2^-3 and 2^-4, 0.14 of it in
    all; an orthogonal factor is the direction of steepest descent, so a
    perturbation e of it costs e^2 of the descent: 0.02 of what the loss fell by."""
    sizes = dict(tokens=1024, inputs=384, outputs=200, steps=25)
    losses = example.train(**sizes)
    exact = plain_losses(rate=0.03, mu=0.9, decay=0.01, seed=0, **sizes)
    assert losses[0] > 0.9                      # the teacher's outputs have unit variance, the weights start at zero
    assert losses[-1] < losses[0]
    for got, want in zip(losses, exact):
        assert abs(got - want) <= 2.0 ** -7 + 0.02 * (exact[0] - want)


def test_gradients_are_the_layer_s(example):
    """Each product against the layer in 64 bits.  A code is off by at most half a
    step of its value (2^-4 in e4m3, 2^-3 in e5m2) or, below the type's normal
    range, by that of its block's smallest normal; the errors of a product's
    terms are independent, so its error is taken against three times the root
    of their squares' sum."""
    import torch
    m, k, n = 700, 300, 260
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    w = torch.randn((n, k), generator=g, device="cuda") / k ** 0.5
    dy = (torch.randn((m, n), generator=g, device="cuda") * 1e-3).bfloat16()
    y, saved = example.forward(x, w)
    momentum = torch.zeros((n, k), device="cuda")
    dx = example.backward(dy, saved, momentum, 0.9)
    torch.cuda.synchronize()
    X, W, D = x.double(), w.double(), dy.double()
    for got, a, b, ha, hb in ((y, X, W.t(), 2.0 ** -4, 2.0 ** -4), (dx, D, W, 2.0 ** -3, 2.0 ** -4),
                              (momentum, D.t(), X, 2.0 ** -3, 2.0 ** -4)):
        want = a @ b
        sigma = ((a.square() @ b.square()) * (ha ** 2 + hb ** 2)).sqrt()
        err = (got.double() - want).abs()
        # (half a step is the largest error, its root mean square is 1/sqrt(3) of it and less)
        assert float((err / (3 * sigma + 2.0 ** -8 * want.abs())).max()) < 1.0
    # beta: the momentum accumulates
    again = momentum.clone()
    example.backward(dy, saved, again, 0.5, need_dx=False)
    assert torch.allclose(again, 1.5 * momentum, rtol=2.0 ** -20, atol=2.0 ** -20 * float(momentum.abs().max()))


def test_step_replays_from_a_graph(example):
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((256, 300), generator=g, device="cuda").bfloat16()
    dy = (torch.randn((256, 200), generator=g, device="cuda") * 1e-3).bfloat16()
    w0 = torch.randn((200, 300), generator=g, device="cuda")
    m0 = torch.randn((200, 300), generator=g, device="cuda") * 1e-3

    def step(w, m):
        y, saved = example.forward(x, w)
        example.backward(dy, saved, m, 0.9)
        example.update(w, m, 0.02, 0.1)
        return y
    wa, ma = w0.clone(), m0.clone()
    for _ in range(3):
        ya = step(wa, ma)
    wb, mb = w0.clone(), m0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        yb = step(wb, mb)
    wb.copy_(w0), mb.copy_(m0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ya, yb) and torch.equal(wa, wb) and torch.equal(ma, mb)
