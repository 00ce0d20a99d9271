"""GPU: the block-scaled product with scales anywhere in fp32's range: neither
the product of a block's two scales nor that of its sum with one of them may
leave the range where the scaled sum itself does not; every form of the kernel
gives the same within the roundings of the definition."""
import numpy as np
import pytest

import mixed_precision_matmul_gb300 as mpg
from fp8_plain import blocks, sum_bound, widen

pytestmark = pytest.mark.gpu

#: forms of the kernel: (rows of A, rows per scale of B, options)
FORMS = {
    "few rows": (7, 128, {}), "few rows, a scale for each row": (50, 1, {}), "few rows, divided": (7, 128, {"splitk": 2}),
    "one CTA": (140, 128, {"cta_pair": -1, "splitk": 1}), "one CTA, columns": (140, 1, {"cta_pair": -1, "splitk": 1}),
    "divided": (140, 128, {"cta_pair": -1, "splitk": 2}), "divided, columns": (140, 1, {"cta_pair": -1, "splitk": 2}),
    "pair": (140, 128, {"cta_pair": 1}), "pair, columns": (140, 1, {"cta_pair": 1}),
}


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


def codes(rows, k, rng, fmt, low, high):
    """Random codes with magnitudes from 2^low to 2^high, in both signs."""
    import torch
    x = 2.0 ** rng.uniform(low, high, (rows, k)) * rng.choice([-1.0, 1.0], (rows, k))
    return torch.from_numpy(x).to(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2)


def run(form, a, sa, b, sb):
    import torch
    m, size, opts = FORMS[form]
    got = mpg.gemm_fp8(a.cuda(), torch.from_numpy(sa).cuda(), b.cuda(), torch.from_numpy(sb).cuda(),
                       out_dtype=torch.float32, opts=mpg.options(**opts)).cpu().double().numpy()
    assert mpg.device_status() == mpg.OK
    wa = widen(a.double().numpy(), sa.astype(np.float64), 1)
    wb = widen(b.double().numpy(), sb.astype(np.float64), size)
    want, den = wa @ wb.T, np.abs(wa) @ np.abs(wb).T
    # below the normal range a rounding is off by half a step of 2^-149: a few for each block
    bound = sum_bound(a.shape[1]) * den + np.abs(want) * 2.0 ** -24 + 4 * blocks(a.shape[1]) * 2.0 ** -149
    return got, want, bound


def check(form, a, sa, b, sb):
    got, want, bound = run(form, a, sa, b, sb)
    assert np.max(np.abs(want)) < 3e38                     # (the case is within fp32's range)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) / np.maximum(bound, 1e-300)))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("ea,eb,low,high", [
    (-70, -70, 6, 8),         # the scales' product is below 2^-126, the result (about 2^-120) is not
    (-125, -14.5, 5, 8),      # and where the scales' product loses bits only
    (-14.5, -125, 5, 8),
    (100, 30, -9, -7),        # the scales' product is above 2^128
    (30, 100, -9, -7),
    (-120, 60, -9, 8), (60, -120, -9, 8),      # a scale and the sum leave the range, the other brings it back
    (-140, 100, -9, 8), (100, -140, -9, 8),    # (a scale below the normal range)
    (-149, 127, -9, 8), (127, -149, -9, 8),
    (115, -100, 4, 8), (-100, 115, 4, 8),
    (90, -30, 4, 8), (88, -149, -9, 8),
])
def test_scales_far_from_one(form, ea, eb, low, high):
    m, size, _ = FORMS[form]
    n, k = 200, 300
    rng = np.random.default_rng(int(1000 + 7 * ea + eb))
    a, b = codes(m, k, rng, "e4m3", low, high), codes(n, k, rng, "e4m3", low, high)
    a[3] = 0                                               # a row of zeros stays one

    def scales(e, rows):
        s = 2.0 ** e * rng.uniform(1.0, 1.9, (rows, blocks(k)))
        return np.maximum(s, 2.0 ** -149).astype(np.float32)
    check(form, a, scales(ea, m), b, scales(eb, -(-n // size)))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scales_of_every_size_in_one_matrix(form, fmt):
    """Rows whose scales are from 2^-149 to 2^127, columns that bring each product near 1."""
    m, size, _ = FORMS[form]
    n, k = 260, 1000
    rng = np.random.default_rng(5)
    top = 8 if fmt == "e4m3" else 15
    a, b = codes(m, k, rng, fmt, -top, top), codes(n, k, rng, fmt, -top, top)
    ea = rng.integers(-149, 128, blocks(k))                # of a block of k: the rows' stay within 2^20 of it
    sa = 2.0 ** np.clip(ea + rng.uniform(-20, 20, (m, blocks(k))), -149, 127)
    sb = 2.0 ** np.clip(-ea + rng.uniform(-20, 20, (-(-n // size), blocks(k))), -149, 127)
    check(form, a, sa.astype(np.float32), b, sb.astype(np.float32))


@pytest.mark.parametrize("form", FORMS)
def test_zeros_under_the_largest_scales_and_infinities(form):
    m, size, _ = FORMS[form]
    n, k = 200, 300
    rng = np.random.default_rng(6)
    a, b = codes(m, k, rng, "e4m3", 0, 8), codes(n, k, rng, "e4m3", 0, 8)
    a[:] = 0
    top = float(np.finfo(np.float32).max)
    sa = np.full((m, blocks(k)), top, np.float32)
    sb = np.full((-(-n // size), blocks(k)), top, np.float32)
    got, _, _ = run(form, a, sa, b, sb)
    assert np.all(got == 0)
    # a scale that is not finite stays in its row
    a = codes(m, k, rng, "e4m3", 0, 8)
    sa = np.ones((m, blocks(k)), np.float32)
    sb = np.ones((-(-n // size), blocks(k)), np.float32)
    sa[2, 1], sa[5, 0] = np.inf, np.nan
    got = run(form, a, sa, b, sb)[0]
    bad = np.zeros((m, n), bool)
    bad[[2, 5]] = True
    assert np.array_equal(~np.isfinite(got), bad)


@pytest.mark.parametrize("pair", [-1, 1])
@pytest.mark.parametrize("k", [100, 900])
def test_a_few_columns_far_from_the_others(pair, k):
    """More tiles than SMs, several to each CTA: one column in one block of k has
    a scale that leaves the range, in the first, a middle and the last tiles;
    the tiles before and after it are right too, and those without one have the
    bits that they have when no column is far."""
    import torch
    m, n = 2433, 2561
    rng = np.random.default_rng(7)
    a, b = codes(m, k, rng, "e4m3", -9, 8), codes(n, k, rng, "e4m3", -9, 8)
    sa = (2.0 ** (-60 + rng.uniform(-3, 3, (m, blocks(k))))).astype(np.float32)
    sb = (2.0 ** (60 + rng.uniform(-3, 3, (n, blocks(k))))).astype(np.float32)
    far = sb.copy()
    last = blocks(k) - 1
    for c, e in ((7, 115), (700, -120), (1500, 118), (1501, 0), (2560, 110)):
        far[c, min(c % 3, last)] = 2.0 ** e * 1.3
    A, SA, B = a.cuda(), torch.from_numpy(sa).cuda(), b.cuda()
    plain, got = (mpg.gemm_fp8(A, SA, B, torch.from_numpy(s).cuda(), out_dtype=torch.float32, opts=mpg.options(cta_pair=pair))
                  for s in (sb, far))
    assert mpg.device_status() == mpg.OK
    wa, wb = widen(a.double().numpy(), sa.astype(np.float64), 1), widen(b.double().numpy(), far.astype(np.float64), 1)
    want, den = wa @ wb.T, np.abs(wa) @ np.abs(wb).T
    bound = sum_bound(k) * den + np.abs(want) * 2.0 ** -24 + 4 * blocks(k) * 2.0 ** -149
    err = np.abs(got.cpu().double().numpy() - want)
    assert np.max(np.abs(want)) < 3e38 and np.all(err <= bound), float(np.max(err / bound))
    tile = 256
    touched = {c // tile for c in (7, 700, 1500, 2560)}
    for t in range(-(-n // tile)):
        if t not in touched:
            assert torch.equal(got[:, t * tile:(t + 1) * tile], plain[:, t * tile:(t + 1) * tile])


@pytest.mark.parametrize("form", FORMS)
def test_scales_of_zero(form):
    """Blocks that a caller's own quantiser gave the scale 0: their sums count nothing, the other rows and
    columns keep their bits."""
    m, size, _ = FORMS[form]
    n, k = 300, 500
    rng = np.random.default_rng(8)
    a, b = codes(m, k, rng, "e4m3", -9, 8), codes(n, k, rng, "e4m3", -9, 8)
    sa = (2.0 ** rng.uniform(-8, 8, (m, blocks(k)))).astype(np.float32)
    sb = (2.0 ** rng.uniform(-8, 8, (-(-n // size), blocks(k)))).astype(np.float32)
    before = run(form, a, sa, b, sb)[0]
    za, zb = sa.copy(), sb.copy()
    za[::3] = 0
    za[1, 2] = 0
    zb[1] = 0
    got, want, bound = run(form, a, za, b, zb)
    assert np.all(np.abs(got - want) <= bound)
    assert np.all(got[::3] == 0) and np.all(got[:, size:2 * size] == 0)
    rows = [r for r in range(m) if r % 3 and r != 1]
    cols = [c for c in range(n) if c // size != 1]
    assert np.array_equal(got[np.ix_(rows, cols)], before[np.ix_(rows, cols)])
