"""GPU: tiles split along k behind whole rounds of tiles, in every epilogue.  Sizes whose last round holds one to
three tiles (152 CTAs, 76 pairs of them): their blocks of k are fewer than the workers.  The workspace holds NaN
before each call, so that a part that nothing wrote shows, and results are the same whatever it held."""
import ctypes

import pytest

import mixed_precision_matmul_gb300 as mpg

torch = pytest.importorskip("torch")
import fused_plain as plain  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"bf16": mpg.BF16, "fp16": mpg.F16}


def normal(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(rows, cols, device="cuda", generator=g)).to(TYPES[dtype])


def twice(size, desc, call):
    """call(workspace, bytes) with a workspace of NaN and with one of zeros: the same bits; the first's results."""
    need = int(size(ctypes.byref(desc)))
    results = []
    for fill in (0xFF, 0):
        ws = torch.full((max(need, 16),), fill, dtype=torch.uint8, device="cuda")
        results.append([t.clone() if t is not None else None for t in call(ws.data_ptr(), need)])
        torch.cuda.synchronize()
        assert mpg.device_status() == mpg.OK
    for a, b in zip(*results):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return results[0]


# (77 and 153 pairs' tiles, 154 of single CTAs: one or two behind whole rounds; the last: 58 of 134)
GATED = [(64, 2048, 9856, "bf16"), (256, 4096, 9856, "fp16"), (2183, 2420, 2131, "bf16"), (100, 4096, 9800, "fp16")]


def layer(t, h, i, dtype):
    x, wg, wu = normal(t, h, dtype, 1), normal(i, h, dtype, 2, h ** -0.5), normal(i, h, dtype, 3, h ** -0.5)
    return x, wg, wu, mpg.GatedLayer(t, h, i, CODES[dtype], 0, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), h, h, h)


@pytest.mark.parametrize("t,h,i,dtype", GATED)
def test_gated_product(t, h, i, dtype):
    x, wg, wu, desc = layer(t, h, i, dtype)
    kept = torch.int16 if dtype == "bf16" else x.dtype
    y, a, b = (torch.empty(t, i, dtype=d, device="cuda") for d in (x.dtype, kept, kept))

    def call(ws, n):
        mpg.gated_gemm_raw(desc, y.data_ptr(), i, a.data_ptr(), i, b.data_ptr(), i, ws, n)
        return y, a, b
    outs = twice(mpg.lib().mpg_gated_gemm_workspace_size, desc, call)
    (ry, ra, rb), (ey, ea, eb) = plain.gated(x, wg, wu, "silu")
    plain.check(outs[0], ry, ey)
    plain.check_kept(outs[1], ra, ea)
    plain.check_kept(outs[2], rb, eb)


@pytest.mark.parametrize("t,h,i,dtype", GATED + [(1792, 2816, 1536, "bf16"), (1790, 2813, 1530, "fp16"), (2304, 4352, 2048, "fp16")])
@pytest.mark.parametrize("need", ["dx", "dw", "both"])
def test_gated_gradients(t, h, i, dtype, need):
    """Recomputed projections; then dX alone, dWg and dWu alone, or all."""
    x, wg, wu, desc = layer(t, h, i, dtype)
    dy = normal(t, i, dtype, 4, 0.1)
    outs = [torch.empty_like(m) if need in (n, "both") else None for m, n in ((x, "dx"), (wg, "dw"), (wu, "dw"))]

    def call(ws, n):
        mpg.gated_gemm_backward_raw(desc, dy.data_ptr(), i, 0, 0, 0, 0,
                                    *(v for o in outs for v in ((o.data_ptr(), h) if o is not None else (0, 0))), ws, n)
        return outs
    got = twice(mpg.lib().mpg_gated_gemm_backward_workspace_size, desc, call)
    for o, r, e in zip(got, *plain.gated_gradients(dy, x, wg, wu, "silu")):
        if o is not None:
            plain.check(o, r, e)


# (153 and 459 tiles of single CTAs, 1825, 154 and 78 of pairs)
LOSS = [(64, 2048, 19500, "bf16"), (120, 2304, 58752, "fp16"), (1092, 2752, 93248, "bf16"), (500, 4096, 19700, "fp16")]


def vocabulary(t, h, v, dtype):
    x, w = normal(t, h, dtype, 5), normal(v, h, dtype, 6, 2 * h ** -0.5)
    target = torch.randint(0, v, (t,), device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    target[::5] = -100
    target[1] = v - 1
    return x, w, target, mpg.VocabLoss(t, h, v, CODES[dtype], x.data_ptr(), w.data_ptr(), h, h, target.data_ptr(), 8, 1, -100)


@pytest.mark.parametrize("t,h,v,dtype", LOSS)
def test_loss(t, h, v, dtype):
    x, w, target, desc = vocabulary(t, h, v, dtype)
    loss, lse = (torch.empty(t, device="cuda") for _ in range(2))

    def call(ws, n):
        mpg.linear_cross_entropy_raw(desc, loss.data_ptr(), lse.data_ptr(), ws, n)
        return loss, lse
    outs = twice(mpg.lib().mpg_linear_cross_entropy_workspace_size, desc, call)
    for o, r, e in zip(outs, *plain.loss(x, w, target)):
        plain.check(o, r, e)


@pytest.mark.parametrize("t,h,v,dtype", LOSS[:2] + [LOSS[3], (1792, 2816, 2999, "bf16"), (3001, 2816, 1790, "fp16")])
@pytest.mark.parametrize("need", ["dx", "dw", "both"])
def test_loss_gradients(t, h, v, dtype, need):
    x, w, target, desc = vocabulary(t, h, v, dtype)
    lse = torch.logsumexp(x.double() @ w.double().t(), 1).float()
    dloss = torch.rand(t, device="cuda", generator=torch.Generator("cuda").manual_seed(8)) + 0.1
    outs = [torch.empty_like(m) if need in (n, "both") else None for m, n in ((x, "dx"), (w, "dw"))]

    def call(ws, n):
        mpg.linear_cross_entropy_backward_raw(desc, lse.data_ptr(), dloss.data_ptr(), 1,
                                              *(v for o in outs for v in ((o.data_ptr(), h) if o is not None else (0, 0))), ws, n)
        return outs
    got = twice(mpg.lib().mpg_linear_cross_entropy_backward_workspace_size, desc, call)
    for o, r, e in zip(got, *plain.loss_gradients(x, w, target, lse, dloss)):
        if o is not None:
            plain.check(o, r, e)
