"""Plain forms of the 8-bit operators in 64 bits, on the CPU, for the tests."""
import numpy as np

BLOCK = 128
TOP = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}   # largest value, fraction bits, smallest normal exponent


def blocks(n):
    return -(-n // BLOCK)


def quantize(x: np.ndarray, fmt: str, rows: int):
    """(values of the codes, scales) of x (float64) with blocks of `rows` x 128,
    by loops over blocks and the definition's own words."""
    top, frac, low = TOP[fmt]
    m, n = x.shape
    q = np.zeros((m, n))
    s = np.ones((-(-m // rows), blocks(n)))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            b = x[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
            fin = np.isfinite(b)
            a = np.max(np.abs(b[fin]), initial=0.0)
            if a > 0:
                t = -126
                if a > top * 2.0 ** -126:
                    t = int(np.floor(np.log2(a / top))) - 1
                    while a > top * 2.0 ** t:
                        t += 1
                s[i, j] = 2.0 ** max(t, -126)
            v = np.where(fin, b, 0.0) / s[i, j]
            e = np.maximum(np.frexp(v)[1] - 1, low)
            step = 2.0 ** (e - frac).astype(np.float64)
            q[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK] = np.where(fin, np.rint(v / step) * step, np.nan)
    return q, s


def widen(q: np.ndarray, s: np.ndarray, rows: int) -> np.ndarray:
    """The values that codes and scales stand for."""
    i = np.arange(q.shape[0]) // rows
    j = np.arange(q.shape[1]) // BLOCK
    return q * s[i][:, j]


# Largest relative error of the product against 64 bits, as a multiple of sum |a b|: the tensor core adds the 128
# products of a block (exact in fp32) with at most one fp32 step (2^-23) each; the scale of a block is one rounding
# and its product with a sum at most two more; the running sum is one rounding a block, and alpha, beta one each.
def sum_bound(k: int) -> float:
    return BLOCK * 2.0 ** -23 + (blocks(k) + 8 + 5) * 2.0 ** -24


HALF_STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
