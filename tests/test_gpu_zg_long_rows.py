"""GPU: logits of long rows of positive products, where sums that are cut off towards zero drift the most."""
import pytest

import mixed_precision_matmul_gb300 as mpg

torch = pytest.importorskip("torch")
import fused_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 7, 16, 17, 130])
@pytest.mark.parametrize("h", [8200, 20000, 65536, 70003])
def test_loss(t, h):
    """The tensor cores sum at most 1024 products at a time (68 units of 2^-23 of their absolute values, as in
    fused_plain); those sums are added in fp32: up to 16 tokens h / 8192 + 1 in each of 8 warps and 8 of the warps',
    beyond h / 1024 + 1, 2^-24 each."""
    g = torch.Generator("cuda").manual_seed(h + t)
    x = torch.rand(t, h, device="cuda", generator=g).bfloat16()
    w = (32 / h * torch.rand(203, h, device="cuda", generator=g)).bfloat16()
    target = torch.randint(0, 203, (t,), device="cuda", generator=g)
    value, lse = mpg.linear_cross_entropy(x, w, target)
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK
    l = x.double() @ w.double().t()                  # (all positive: the sums of absolute values too)
    adds = h / 8192 + 10 if t <= 16 else h / 1024 + 2
    top = l.amax(dim=1)
    ref = torch.logsumexp(l, dim=1)
    e = (68 * 2.0 ** -23 + adds * 2.0 ** -24) * top + 3 * 2.0 ** -24 * top + 2.0 ** -22 + 20 * 2.0 ** -24 * (1 + ref)
    plain.check(lse, ref, e)
    plain.check(value, ref - l.gather(1, target[:, None])[:, 0], 2 * e)
