"""GPU: gradients of the gated product in fp16 whose factors up act'(gate) and act(gate) are far above 2^11, or far
below 1: the scale that dgate and dup carry comes from themselves then."""
import pytest

import mixed_precision_matmul_gb300 as mpg

torch = pytest.importorskip("torch")
import fused_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK


def normal(rows, cols, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(rows, cols, device="cuda", generator=g)).half()


def layer(t, h, i):
    """Normal values, but for a token with an input channel of 120, and inner values that it meets: an up of 9600 at a
    gate of 120 (dgate = 9600 dY), and a gate of 9600 at an up of 120 (dup = 9600 dY).  dY is largest there, 2^-7."""
    x, wg, wu, dy = normal(t, h, 1), normal(i, h, 2, h ** -0.5), normal(i, h, 3, h ** -0.5), normal(t, i, 4, 2.0 ** -11)
    x[t // 2, 0] = 120.0
    a, b = i // 3, i - 1
    wg[a], wu[a], wg[b], wu[b] = 0, 0, 0, 0
    wg[a, 0], wu[a, 0], wg[b, 0], wu[b, 0] = 1.0, 80.0, 80.0, 1.0
    dy[t // 2, a] = dy[t // 2, b] = 2.0 ** -7
    return x, wg, wu, dy


def references(dy, x, wg, wu, act, kept):
    """fused_plain's, but for what subnormal dgate and dup leave: half of 2^-24 where the largest of them is 2^14 at
    least, so 2^-39 of the largest, in the place of 2^-29 of the largest dY."""
    refs, bounds = plain.gated_gradients(dy, x, wg, wu, act, kept)
    d = dy.double()
    if kept is None:
        a, s = plain.act(x.double() @ wg.double().t(), act)
        b = x.double() @ wu.double().t() * s
    else:
        a, b = (plain.kept_values(k) for k in kept)
    more = float(torch.maximum((d * a).abs().max(), (d * b).abs().max())) * 2.0 ** -39 - float(d.abs().max()) * 2.0 ** -29
    sums = (wg.double().abs().sum(0) + wu.double().abs().sum(0), x.double().abs().sum(0), x.double().abs().sum(0))
    return refs, [e + more * s[None] for e, s in zip(bounds, sums)]


# few rows, single CTAs, pairs, split tiles and their joining launch, split tiles behind whole rounds
SHAPES = [(5, 64, 200), (16, 1000, 77), (70, 72, 264), (600, 520, 1500), (40, 4000, 70), (600, 4096, 515), (64, 2048, 9856)]


@pytest.mark.parametrize("t,h,i", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_large_factors(t, h, i, act):
    x, wg, wu, dy = layer(t, h, i)
    _, a, b = mpg.gated_gemm(x, wg, wu, act=act, keep=True)
    assert float(b.abs().max()) >= 9000 and float(a.abs().max()) >= 9000
    for kept in (None, (a, b)):
        refs, bounds = references(dy, x, wg, wu, act, kept)
        outs = mpg.gated_gemm_backward(dy, x, wg, wu, act=act, kept=kept)
        ok()
        for o, r, e in zip(outs, refs, bounds):
            assert float(r.abs().max()) < 60000
            plain.check(o, r, e)


@pytest.mark.parametrize("t,h,i", SHAPES)
def test_small_factors(t, h, i):
    """Gates and ups of 2^-13: dgate and dup are 2^-14 of dY, and keep fp16's precision all the same."""
    x, wg, wu, dy = normal(t, h, 5, 2.0 ** -10), normal(i, h, 6, 2.0 ** -3 * h ** -0.5), normal(i, h, 7, 2.0 ** -3 * h ** -0.5), normal(t, i, 8)
    refs, bounds = references(dy, x, wg, wu, "silu", None)
    outs = mpg.gated_gemm_backward(dy, x, wg, wu)
    ok()
    for o, r, e in zip(outs, refs, bounds):
        plain.check(o, r, e)


@pytest.mark.parametrize("t,h,i", SHAPES[:5])
def test_an_infinite_gradient_beside_large_factors(t, h, i):
    """A token whose dY is infinite has gradients that are no numbers; the other tokens' dX are those without it."""
    x, wg, wu, dy = layer(t, h, i)
    dy[0, 1] = float("inf")
    others = torch.arange(t, device="cuda") != 0
    quiet = torch.where(others[:, None], dy, 0)
    # (dY itself is not scaled: what is below fp16's normal numbers is off by 2^-25 at most)
    for kept in (None, mpg.gated_gemm(x, wg, wu, keep=True)[1:]):
        refs, bounds = references(quiet, x, wg, wu, "silu", kept)
        dx, _, _ = mpg.gated_gemm_backward(dy, x, wg, wu, kept=kept)
        ok()
        assert not dx[0].isfinite().any()
        floor = 2.0 ** -25 * (wg.double().abs().sum(0) + wu.double().abs().sum(0))
        plain.check(dx[others], refs[0][others], bounds[0][others] + floor[None])


@pytest.mark.parametrize("t", [5, 70, 600])
def test_a_graph_over_inputs_of_both_kinds(t):
    """Captured once; replayed with factors that fit the first scale, that do not, and that do again."""
    x, wg, wu, dy = layer(t, 520, 300)
    graph = torch.cuda.CUDAGraph()
    mpg.gated_gemm_backward(dy, x, wg, wu)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = mpg.gated_gemm(x, wg, wu, keep=True)[1:]
        couts = (*mpg.gated_gemm_backward(dy, x, wg, wu), *mpg.gated_gemm_backward(dy, x, wg, wu, kept=kept))
    large, usual = x.clone(), normal(t, 520, 9)
    for inputs in (usual, large, usual):
        x.copy_(inputs)
        graph.replay()
        torch.cuda.synchronize()
        k = mpg.gated_gemm(x, wg, wu, keep=True)[1:]
        refs = (*mpg.gated_gemm_backward(dy, x, wg, wu), *mpg.gated_gemm_backward(dy, x, wg, wu, kept=k))
        assert all(torch.equal(a, b) for a, b in zip(couts, refs)) and all(o.isfinite().all() for o in refs)
    ok()
