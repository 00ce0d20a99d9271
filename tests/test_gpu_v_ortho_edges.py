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
