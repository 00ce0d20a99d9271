"""GPU: the orthogonalised update where it can go wrong beside its sizes: shares
of a divided tile that hold few rows or none."""
import pytest

import mixed_precision_matmul_gb300 as mpg
from test_gpu_t_ortho import exact, momentum, rounded, tdtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


@pytest.mark.parametrize("m,n", [(100, 576), (33, 2000), (2000, 33), (130, 1000), (260, 1030), (7, 640)])
def test_divided_tiles_with_rows_beyond_the_matrix(m, n):
    """Few tiles: k divided among the CTAs of a cluster, each with a share of the
    tile's rows, of which the last ones lie beyond the matrix.  No CTA may leave
    while another reads its sums: many calls in a row give the same bits, and
    those are the 64-bit result's within twice what its storage costs."""
    import torch
    gs = [momentum(1, m, n, seed, "bf16").cuda() for seed in (m, n + 1)]
    first = [mpg.orthogonalize(g, out_dtype=tdtype("fp32")) for g in gs]
    for g, f in zip(gs, first):
        want, sim = exact(g.cpu(), 5), rounded(g.cpu(), 5).double()
        norm = want.norm()
        assert (f.cpu().double() - want).norm() / norm <= 2 * (sim - want).norm() / norm + 1e-5
    outs = [mpg.orthogonalize(gs[i & 1], out_dtype=tdtype("fp32")) for i in range(60)]
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK
    assert all(torch.equal(o, first[i & 1]) for i, o in enumerate(outs))


def stored(x):
    """Rounded to fp16's 11 bits, of any exponent."""
    import torch
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0 ** 11), e - 11)


def rounded_at_any_scale(g, steps, eps):
    """The operator's roundings with X stored times whatever power of two suits it; S and b S + c S S in fp16."""
    a, b, c = mpg.NS_COEFFS
    x = g.double()
    x = stored(x) / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + eps)
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    for i in range(steps):
        s = (x @ x.mT).half().double()
        y = a * x + (b * s + c * (s @ s)).half().double() @ x
        x = stored(y) if i + 1 < steps else y
    return x.mT if tall else x


def of_norm(b, m, n, seed, dtype, norm):
    g = momentum(b, m, n, seed, "fp32").double()
    return (g / g.square().sum(dim=(1, 2), keepdim=True).sqrt() * norm).to(tdtype(dtype))


def check_small(g, steps, eps, **kw):
    """Against 64 bits within twice the storage's own roundings; elements far below the others of a matrix
    lose 2^-25 of its scale a step, less than 1e-5 of the norm up to 100 rows and 9 steps."""
    got = mpg.orthogonalize(g.cuda(), steps=steps, eps=eps, out_dtype=tdtype("fp32"), **kw).cpu().double()
    assert mpg.device_status() == mpg.OK
    want, sim = exact(g, steps, eps), rounded_at_any_scale(g, steps, eps)
    for o, w, s in zip(got, want, sim):
        assert (o - w).norm() <= (2 * (s - w).norm() / w.norm() + 1e-5) * w.norm(), float((o - w).norm() / w.norm())


@pytest.mark.parametrize("b,m,n,dtype", [(1, 100, 256, "bf16"), (2, 64, 500, "fp32"), (1, 500, 64, "bf16"), (1, 1, 40, "fp16")])
@pytest.mark.parametrize("steps", [1, 2, 5, 9])
@pytest.mark.parametrize("norm,eps", [(1e-8, 1e-7), (1e-10, 1e-7), (1e-12, 1e-7), (1e-13, 1e-7), (1e-14, 1e-7), (1e-20, 1e-7),
                                      (1e-27, 1e-7), (1e-20, 1.0), (1e-4, 1e28), (3.0, 1e5), (1e3, 2e3)])
def test_norms_far_below_eps(b, m, n, dtype, steps, norm, eps):
    if dtype == "fp16" and norm < 1e-6:
        pytest.skip("below fp16's range")
    check_small(of_norm(b, m, n, m + steps, dtype, norm), steps, eps)


def test_each_matrix_of_a_batch_has_its_own_norm():
    import torch
    norms = [1.0, 1e-6, 1e-12, 1e-25, 1e4, 3e-8]
    g = torch.cat([of_norm(1, 90, 200, i, "bf16", v) for i, v in enumerate(norms)])
    check_small(g, 5, 1e-7)
    # and the power of two of a small matrix and eps changes no bit
    base = mpg.orthogonalize(g.cuda(), eps=1e-7, out_dtype=tdtype("fp32"))
    for e in (-7, -3, 25):
        assert torch.equal(g * 2.0 ** e * 2.0 ** -e, g)       # (exact in bf16)
        assert torch.equal(base, mpg.orthogonalize(g.cuda() * 2.0 ** e, eps=float(torch.tensor(1e-7)) * 2.0 ** e,
                                                   out_dtype=tdtype("fp32")))


def test_small_updates_folded_into_a_weight():
    """alpha brings a small update back: the weight's change is the update's, within its own roundings."""
    import torch
    g = of_norm(1, 90, 200, 3, "bf16", 1e-12)
    w = torch.randn((1, 90, 200), generator=torch.Generator().manual_seed(1))
    o = w.cuda()
    mpg.orthogonalize(g.cuda(), O=o, eps=1e-7, alpha=-4096.0, beta=0.5)
    want = 0.5 * w.double() - 4096.0 * exact(g, 5, 1e-7)
    part = 4096.0 * exact(g, 5, 1e-7)
    sim = (rounded_at_any_scale(g, 5, 1e-7) * 4096.0 - part).norm() / part.norm()
    # (the weights' rounding: half a step of each, 2^-24)
    assert (o.cpu().double() - want).norm() <= (2 * sim + 1e-5) * part.norm() + 2.0 ** -23 * w.double().norm()


@pytest.mark.parametrize("eps", [1e-7, 1e-20, 1e-30, 1e-38, 1e-44])
@pytest.mark.parametrize("shape", [(3, 40, 50), (2, 300, 200), (2, 1, 1)])
def test_zero_matrices_stay_zero_with_any_eps(eps, shape):
    """0 / (0 + eps) is 0, and a weight that takes the update keeps its own."""
    import torch
    g = torch.randn(shape, generator=torch.Generator().manual_seed(1)).cuda()
    g[0] = 0
    o = mpg.orthogonalize(g, eps=eps, out_dtype=tdtype("fp32"))
    assert (o[0] == 0).all() and torch.isfinite(o).all() and (o[1] != 0).any()
    w = torch.randn(shape, generator=torch.Generator().manual_seed(2)).cuda()
    w0 = w.clone()
    mpg.orthogonalize(g, O=w, eps=eps, alpha=-0.1, beta=0.5)
    assert torch.equal(w[0], 0.5 * w0[0]) and torch.isfinite(w).all()


@pytest.mark.parametrize("b,m,n", [(4, 70, 96), (3, 130, 65), (2, 300, 260)])
def test_matrices_beside_one_another(b, m, n):
    """The blocks of columns of one wide weight as a batch, in and out, without touching what lies between."""
    import torch
    g = momentum(b, m, n, 9, "bf16").cuda()
    want = mpg.orthogonalize(g, out_dtype=tdtype("fp32"))
    wide_g = torch.full((m, b, n + 3), 7.0, dtype=g.dtype, device="cuda")
    wide_g[:, :, :n] = g.permute(1, 0, 2)
    wide_o = torch.full((m, b, n + 3), 7.0, device="cuda")
    o = wide_o[:, :, :n].permute(1, 0, 2)
    mpg.orthogonalize(wide_g[:, :, :n].permute(1, 0, 2), O=o)
    assert torch.equal(o, want)
    assert (wide_o[:, :, n:] == 7.0).all()


@pytest.mark.parametrize("norm", [1e-36, 1e-39, 3e-42])
@pytest.mark.parametrize("eps", [0.0, 1e-40])
def test_norms_below_the_normal_range(norm, eps):
    """fp32 gradients of subnormal size: every bit that they still have counts."""
    import torch
    eps = float(torch.tensor(eps))                             # (as the operator receives it)
    g = of_norm(1, 40, 60, 4, "fp32", norm)
    check_small(g, 5, eps)
