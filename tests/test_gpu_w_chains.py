"""GPU: chains of the 8-bit operators and the orthogonalised update over the same
buffers, back to back and with other inputs every time: each kernel may be
resident before the one that writes its inputs has finished, and must not see
what the buffers held before."""
import pytest

import mixed_precision_matmul_gb300 as mpg

pytestmark = pytest.mark.gpu

ROUNDS = 24


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


def inputs(shape, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    # (each round's values have a size of their own, so that scales and norms differ)
    return [torch.randn(shape, generator=g, device="cuda") * 2.0 ** (3 * (i % 5)) for i in range(ROUNDS)]


@pytest.mark.parametrize("m,n,k,pad,opts", [
    (3, 640, 1024, 0, None), (40, 300, 1024, 0, None),                     # few rows
    (300, 260, 640, 0, {"cta_pair": -1}), (300, 260, 640, 0, {"cta_pair": 1}),
    (200, 256, 2048, 0, {"splitk": 4, "tile_n": 128}),
    (70, 200, 515, 3, None),                                               # lines off 16 bytes: copied first
])
def test_quantised_operands_in_the_same_buffers(m, n, k, pad, opts):
    import torch
    xs, ws = inputs((m, k), 1), inputs((n, k), 2)
    ld, kb = k + pad if pad else (k + 15) // 16 * 16, (k + 127) // 128
    aq = torch.empty((m, ld), dtype=torch.uint8, device="cuda")
    bq = torch.empty((n, ld), dtype=torch.uint8, device="cuda")
    sa = torch.empty((kb, m), device="cuda")
    sb = torch.empty(((n + 127) // 128, kb), device="cuda")
    A = aq[:, :k].view(torch.float8_e4m3fn)
    B = bq[:, :k].view(torch.float8_e4m3fn)
    cs = [torch.empty((m, n), device="cuda") for _ in range(ROUNDS)]
    o = mpg.options(**opts) if opts else None
    want = [mpg.gemm_fp8(*mpg.fp8_quantize(x), *mpg.fp8_quantize(w, block="tile"), out_dtype=torch.float32, opts=o)
            for x, w in zip(xs, ws)]
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    for x, w, c in zip(xs, ws, cs):
        mpg.fp8_quantize_raw(n, k, w.data_ptr(), k, mpg.F32, mpg.E4M3, 128, bq.data_ptr(), ld, sb.data_ptr(), kb, 1, 0, 0,
                             0, 0, 0, stream)
        mpg.fp8_quantize_raw(m, k, x.data_ptr(), k, mpg.F32, mpg.E4M3, 1, aq.data_ptr(), ld, sa.data_ptr(), 1, m, 0, 0,
                             0, 0, 0, stream)
        mpg.gemm_fp8(A, sa.t(), B, sb, C=c, opts=o)
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK
    for c, w in zip(cs, want):
        assert torch.equal(c, w)


@pytest.mark.parametrize("shape", [(1, 90, 300), (1, 300, 130), (8, 512, 512), (30, 256, 300)])
def test_updates_of_a_momentum_that_the_product_writes(shape):
    """A product writes the matrix that the next launch takes the norm of; the
    workspace, the factors and the iterates are in the same places every time."""
    import torch
    b, m, n = shape
    k = 256
    xs, ds = inputs((b * m, k), 3), inputs((n, k), 4)
    qs = [(mpg.fp8_quantize(x), mpg.fp8_quantize(d)) for x, d in zip(xs, ds)]
    M = torch.empty((b * m, n), device="cuda")
    ws = torch.empty(mpg.orthogonalize_workspace_size(m, n, b), dtype=torch.uint8, device="cuda")
    want = []
    for x, d in qs:
        mpg.gemm_fp8(*x, *d, C=M)
        torch.cuda.synchronize()
        want.append(mpg.orthogonalize(M.view(shape), out_dtype=torch.float32))
        torch.cuda.synchronize()
    outs = [torch.empty(shape, device="cuda") for _ in range(ROUNDS)]
    torch.cuda.synchronize()
    for (x, d), o in zip(qs, outs):
        mpg.gemm_fp8(*x, *d, C=M)
        mpg.orthogonalize(M.view(shape), O=o, workspace=ws)
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
