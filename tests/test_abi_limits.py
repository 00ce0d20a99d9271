"""CPU: the largest extents of the 8-bit operators and the orthogonalised update.
Their kernels count rows and columns in 32 bits, to the end of the last tile of
256; what does not fit is refused on the host before a launch."""
import ctypes

import pytest

import mixed_precision_matmul_gb300 as mpg

TOP = 2 ** 31 - 256


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


@pytest.mark.parametrize("size", [TOP + 1, TOP + 128, 2 ** 31 - 1])
def test_extents_whose_last_tile_leaves_32_bits_are_refused(size):
    def quantize(rows, cols):
        return mpg.fp8_quantize_raw(rows, cols, 4096, cols, mpg.F32, mpg.E4M3, 1, 4096, cols, 4096, 1, rows, 0, 0, 0, 1, 1,
                                    check=False)

    def product(m, n, k):
        a, b = (mpg.Fp8Operand(4096, k, 0, 1, 4096, 1, 1) for _ in range(2))
        return mpg.gemm_fp8_raw(m, n, k, a, b, 4096, n, 1.0, 0.0, check=False)

    def update(m, n):
        return mpg.orthogonalize_raw(m, n, 1, 4096, n, 0, mpg.BF16, 4096, n, 0, mpg.BF16, workspace=4096,
                                     workspace_bytes=2 ** 62, check=False)
    for status in (quantize(1, size), quantize(size, 1), product(size, 1, 16), product(1, size, 16), product(1, 1, size),
                   update(size, 1), update(1, size)):
        assert status == mpg.ERR_INVALID_ARG
        assert "2^31-256" in mpg.last_error()


def test_workspace_queries_end_where_the_operators_do():
    odd = mpg.Fp8Operand(4097, 17, 0, 1, 4096, 1, 1)
    even = mpg.Fp8Operand(4096, 16, 0, 1, 4096, 1, 1)
    size = mpg.lib().mpg_gemm_fp8_workspace_size
    assert size(TOP, 5, 16, ctypes.byref(odd), ctypes.byref(even)) == TOP * 16
    assert size(TOP + 1, 5, 16, ctypes.byref(odd), ctypes.byref(even)) == 0
    assert mpg.orthogonalize_workspace_size(1, TOP) > 4 * TOP and mpg.orthogonalize_workspace_size(1, TOP + 1) == 0


def orthogonalize(batch, m, n, ldo, stride):
    return mpg.orthogonalize_raw(m, n, batch, 4096, n, 0, mpg.BF16, 4096, ldo, stride, mpg.BF16, workspace=0, check=False)


def test_matrices_of_o_may_lie_beside_one_another():
    """Batches along the columns of one wide matrix do not overlap (what is refused is the missing workspace)."""
    assert orthogonalize(4, 8, 16, 64, 16) == mpg.ERR_WORKSPACE
    assert orthogonalize(4, 8, 16, 70, 18) == mpg.ERR_WORKSPACE
    assert orthogonalize(4, 8, 16, 16, 128) == mpg.ERR_WORKSPACE
    for ldo, stride in ((64, 15), (63, 16), (66, 17), (16, 16), (16, 127)):
        assert orthogonalize(4, 8, 16, ldo, stride) == mpg.ERR_INVALID_ARG
        assert "overlap" in mpg.last_error()
