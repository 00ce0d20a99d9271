"""GPU: the gated product, the vocabulary's loss, clipping and the orthogonalised
update together, as the example runs them: its gradients against 64 bits, and a
step's work captured and replayed."""
import importlib.util
import os

import pytest

import mixed_precision_matmul_gb300 as mpg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    mpg.build()
    spec = importlib.util.spec_from_file_location("gated_lm_step", os.path.join(ROOT, "examples", "gated_lm_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def exact_gradients(x, target, weights, ignore):
    """The same by autograd in 64 bits."""
    leaves = [t.double().requires_grad_(True) for t in (x, *weights)]
    a, wg, wu, wd, wv = leaves
    gate = a @ wg.t()
    h = (gate * torch.sigmoid(gate) * (a @ wu.t())) @ wd.t()
    loss = torch.nn.functional.cross_entropy(h @ wv.t(), target, ignore_index=ignore)
    return float(loss.detach()), torch.autograd.grad(loss, leaves)


@pytest.mark.parametrize("tokens,hidden,inner,vocab,dtype", [
    (300, 136, 264, 1003, torch.bfloat16), (300, 136, 264, 1003, torch.float16), (77, 65, 129, 515, torch.bfloat16),
    (12, 128, 256, 4099, torch.float16), (2048, 256, 704, 5000, torch.bfloat16)])
def test_gradients_are_the_formulas(example, tokens, hidden, inner, vocab, dtype):
    """On no way from the inputs to a gradient are there more than twelve roundings to 16 bits
    (y, h, D, dh, dy, what is kept, dgate or dup, the result; dy's and D's own operands
    again).  Each is half a step of the value at most, and a product of independent matrices
    carries such a part of its operand's norm into the same part of its result's."""
    x, target, weights, _ = example.draw(tokens, hidden, inner, vocab, dtype=dtype)
    loss, grads = example.gradients(x, target, *weights)
    assert mpg.device_status() == mpg.OK
    ref, refs = exact_gradients(x, target, weights, example.IGNORE)
    step = torch.finfo(dtype).eps / 2
    assert abs(float(loss) - ref) <= 12 * step * ref
    for g, r in zip(grads, refs):
        # (fp16's smallest numbers: a gradient of a mean has elements below them)
        least = 2.0 ** -25 * r.numel() ** 0.5 * 4 if dtype == torch.float16 else 0.0
        assert float((g.double() - r).norm()) <= 12 * step * float(r.norm()) + least


def test_the_example_runs(example):
    losses = example.train(tokens=512, hidden=128, inner=352, vocab=1000, steps=3)
    assert len(losses) == 3 and all(l == l and l < float("inf") for l in losses)
    assert mpg.device_status() == mpg.OK


def test_a_captured_step_replays(example):
    """A step's work in a graph, while eager results of the same tensors live; replayed with other inputs."""
    x, target, weights, masters = example.draw(400, 128, 352, 1000, seed=3)

    def work():
        loss, grads = example.gradients(x, target, *weights)
        clipped = [torch.empty_like(m) for m in masters]
        norm = mpg.clip_grad_norm(grads[1:], 0.5, out=clipped)
        return [loss, norm, *grads, *clipped]
    eager = work()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, captured))
    x.mul_(0.5)
    weights[0].mul_(2.0)
    target.copy_(target.roll(7))
    again = work()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, captured))
    assert not torch.equal(again[2], eager[2])
    # two graphs that share a pool and their leaves
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second, pool=graph.pool()):
        other = work()
    second.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, other))
    assert mpg.device_status() == mpg.OK
