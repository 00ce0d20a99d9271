"""GPU: the 8-bit torch forms give the same whether their calls are marshalled
by the extension or in Python."""
import pytest

import mixed_precision_matmul_gb300 as mpg
from mixed_precision_matmul_gb300 import fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(1, 300, 256), (70, 129, 515), (300, 260, 640)])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_python_form_is_the_extension_s(m, n, k, block, monkeypatch):
    import torch
    mpg.build()
    assert fp8._calls() is not None
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = (torch.randn(s, generator=g, device="cuda") for s in ((m, k), (n, k)))

    def run():
        q = mpg.fp8_quantize(x.bfloat16(), fmt="e5m2", transpose=True)
        wq, ws = mpg.fp8_quantize(w, block=block)
        y = [mpg.gemm_fp8(q[0], q[1], wq, ws, alpha=0.5, out_dtype=t) for t in (None, torch.float32, torch.float16)]
        odd = mpg.gemm_fp8(q[0][:, 1:k - 1], q[1], wq[:, 1:k - 1], ws)         # off 16 bytes: copied
        return [*q, wq, ws, *y, odd]
    one = run()
    monkeypatch.setattr(fp8, "_calls", lambda: None)
    for a, b in zip(one, run()):
        assert a.dtype == b.dtype and a.stride() == b.stride() and torch.equal(a.float(), b.float())
