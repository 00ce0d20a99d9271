"""CPU: argument checks of mpg_orthogonalize (everything is refused on the host
before a launch), its workspace query, and the refusals of the torch form."""
import pytest

import mixed_precision_matmul_gb300 as mpg


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


def call(m=8, n=16, batch=1, G=4096, ldg=16, sG=0, gdt=mpg.BF16, O=8192, ldo=16, sO=0, odt=mpg.BF16, steps=5,
         coeffs=(1.0, 2.0, 3.0), eps=1e-7, alpha=1.0, beta=0.0, ws=4096, ws_bytes=1 << 30):
    return mpg.orthogonalize_raw(m, n, batch, G, ldg, sG, gdt, O, ldo, sO, odt, steps, coeffs, eps, alpha, beta, ws,
                                 ws_bytes, 0, check=False)


@pytest.mark.parametrize("kw,expect", [
    (dict(m=-1), mpg.ERR_INVALID_ARG),
    (dict(n=2 ** 31), mpg.ERR_INVALID_ARG),
    (dict(batch=-1), mpg.ERR_INVALID_ARG),
    (dict(batch=65536), mpg.ERR_INVALID_ARG),
    (dict(ldg=15), mpg.ERR_INVALID_ARG),
    (dict(ldo=15), mpg.ERR_INVALID_ARG),
    (dict(gdt=3), mpg.ERR_INVALID_ARG),
    (dict(odt=-1), mpg.ERR_INVALID_ARG),
    (dict(steps=0), mpg.ERR_INVALID_ARG),
    (dict(steps=101), mpg.ERR_INVALID_ARG),
    (dict(coeffs=None), mpg.ERR_INVALID_ARG),
    (dict(coeffs=(1.0, float("nan"), 2.0)), mpg.ERR_INVALID_ARG),
    (dict(alpha=float("inf")), mpg.ERR_INVALID_ARG),
    (dict(beta=float("nan")), mpg.ERR_INVALID_ARG),
    (dict(eps=-1.0), mpg.ERR_INVALID_ARG),
    (dict(eps=float("nan")), mpg.ERR_INVALID_ARG),
    (dict(G=0), mpg.ERR_INVALID_ARG),
    (dict(O=0), mpg.ERR_INVALID_ARG),
    (dict(G=4097), mpg.ERR_INVALID_ARG),
    (dict(odt=mpg.F32, O=8194), mpg.ERR_INVALID_ARG),
    (dict(sG=-1), mpg.ERR_INVALID_ARG),
    (dict(batch=2, sO=7 * 16 + 15), mpg.ERR_INVALID_ARG),
    (dict(ws=0), mpg.ERR_WORKSPACE),
    (dict(ws=4097), mpg.ERR_WORKSPACE),
    (dict(ws_bytes=100), mpg.ERR_WORKSPACE),
])
def test_refuses(kw, expect):
    assert call(**kw) == expect
    assert mpg.last_error()


def test_empty_is_a_no_op():
    assert call(m=0) == mpg.OK
    assert call(n=0) == mpg.OK
    assert call(batch=0) == mpg.OK


def test_workspace_size():
    size = mpg.orthogonalize_workspace_size
    assert size(0, 5) == 0 and size(5, 5, 0) == 0 and size(2 ** 31, 5) == 0 and size(5, 5, 65536) == 0
    # two copies of X, S and b S + c S S in fp16, and the norm's partial sums
    m, n, b = 256, 1000, 3
    assert 2 * (2 * b * m * n + 2 * b * m * m) <= size(m, n, b) <= 2 * (2 * b * m * n + 2 * b * m * m) + b * 4096
    assert size(m, n, b) == pytest.approx(size(n, m, b), rel=0.02)
    need = size(8, 16)
    assert call(ws_bytes=need - 1) == mpg.ERR_WORKSPACE


def test_torch_form_refuses():
    import torch
    g = torch.zeros(4, 6)
    with pytest.raises(ValueError):
        mpg.orthogonalize(g)                         # not on a CUDA device
    with pytest.raises(ValueError):
        mpg.orthogonalize(g[0])
    with pytest.raises(TypeError):
        mpg.orthogonalize(g.double())
    with pytest.raises(ValueError):
        mpg.orthogonalize(g, coeffs=(1.0, 2.0))
