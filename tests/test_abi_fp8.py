"""CPU: argument checks of mpg_fp8_quantize and mpg_gemm_fp8 (everything is
refused on the host before a launch), the workspace query, the refusals of the
torch forms, and the plain forms that the GPU tests compare with."""
import numpy as np
import pytest

import mixed_precision_matmul_gb300 as mpg
from fp8_plain import quantize, widen


@pytest.fixture(scope="module", autouse=True)
def built():
    mpg.build()


def q(rows=4, cols=256, X=4096, ldx=256, dt=mpg.F32, fmt=0, sr=1, Q=4096, ldq=256, S=4096, QT=0, ldqt=0, ST=0,
      strides=(1, 4, 1, 1)):
    return mpg.fp8_quantize_raw(rows, cols, X, ldx, dt, fmt, sr, Q, ldq, S, strides[0], strides[1], QT, ldqt, ST,
                                strides[2], strides[3], check=False)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), mpg.ERR_INVALID_ARG),
    (dict(cols=2 ** 31), mpg.ERR_INVALID_ARG),
    (dict(ldx=255), mpg.ERR_INVALID_ARG),
    (dict(dt=3), mpg.ERR_INVALID_ARG),
    (dict(fmt=2), mpg.ERR_UNSUPPORTED),
    (dict(fmt=-1), mpg.ERR_UNSUPPORTED),
    (dict(sr=64), mpg.ERR_UNSUPPORTED),
    (dict(Q=0), mpg.ERR_INVALID_ARG),                       # no form asked for
    (dict(S=0), mpg.ERR_INVALID_ARG),
    (dict(ldq=255), mpg.ERR_INVALID_ARG),
    (dict(QT=4096, ldqt=3, ST=4096), mpg.ERR_INVALID_ARG),
    (dict(QT=4096, ldqt=4), mpg.ERR_INVALID_ARG),           # QT without ST
    (dict(strides=(-1, 4, 1, 1)), mpg.ERR_INVALID_ARG),
    (dict(X=0), mpg.ERR_INVALID_ARG),
    (dict(X=4098), mpg.ERR_INVALID_ARG),                    # fp32 off its element
    (dict(S=4097), mpg.ERR_INVALID_ARG),
])
def test_quantizer_refuses(kw, expect):
    assert q(**kw) == expect
    assert mpg.last_error()


def test_quantizer_empty_is_a_no_op():
    assert q(rows=0) == mpg.OK
    assert q(cols=0) == mpg.OK


def op(data=4096, ld=256, fmt=0, sr=1, scale=4096, rs=1, ks=4):
    return mpg.Fp8Operand(data, ld, fmt, sr, scale, rs, ks)


def g(m=4, n=8, k=256, A=None, B=None, C=4096, ldc=8, opts=None, ws=0, ws_bytes=0, alpha=1.0):
    return mpg.gemm_fp8_raw(m, n, k, A or op(), B or op(sr=128), C, ldc, alpha, 0.0, ws, ws_bytes, 0, opts, check=False)


@pytest.mark.parametrize("kw,expect", [
    (dict(m=-1), mpg.ERR_INVALID_ARG),
    (dict(n=2 ** 31), mpg.ERR_INVALID_ARG),
    (dict(A=op(ld=255)), mpg.ERR_INVALID_ARG),
    (dict(A=op(fmt=2)), mpg.ERR_UNSUPPORTED),
    (dict(B=op(sr=2)), mpg.ERR_UNSUPPORTED),
    (dict(A=op(data=None)), mpg.ERR_INVALID_ARG),
    (dict(B=op(scale=None)), mpg.ERR_INVALID_ARG),
    (dict(B=op(scale=4098)), mpg.ERR_INVALID_ARG),
    (dict(A=op(rs=-1)), mpg.ERR_INVALID_ARG),
    (dict(ldc=7), mpg.ERR_INVALID_ARG),
    (dict(C=0), mpg.ERR_INVALID_ARG),
    (dict(C=4097), mpg.ERR_INVALID_ARG),
])
def test_product_refuses(kw, expect):
    assert g(**kw) == expect
    assert mpg.last_error()


@pytest.mark.parametrize("o,expect", [
    (dict(tile_n=48), mpg.ERR_INVALID_ARG),
    (dict(tile_n=256), mpg.ERR_INVALID_ARG),
    (dict(splitk=9), mpg.ERR_INVALID_ARG),
    (dict(splitk=-1), mpg.ERR_INVALID_ARG),
    (dict(c_dtype=3), mpg.ERR_INVALID_ARG),
    (dict(cta_pair=2), mpg.ERR_INVALID_ARG),
    (dict(cta_pair=1, tile_n=128), mpg.ERR_INVALID_ARG),
    (dict(cta_pair=1, splitk=2), mpg.ERR_INVALID_ARG),
    (dict(wait_timeout_ns=-1), mpg.ERR_INVALID_ARG),
])
def test_product_refuses_options(o, expect):
    assert g(opts=mpg.options(**o)) == expect


def test_product_null_description():
    assert mpg.gemm_fp8_raw(4, 8, 256, None, op(), 4096, 8, 1.0, 0.0, check=False) == mpg.ERR_INVALID_ARG


def test_product_empty_is_a_no_op():
    assert g(m=0) == mpg.OK
    assert g(n=0) == mpg.OK


def test_workspace_covers_what_tma_cannot_describe():
    import ctypes
    size = mpg.lib().mpg_gemm_fp8_workspace_size

    def need(m, n, k, a, b):
        return size(m, n, k, ctypes.byref(a), ctypes.byref(b))
    assert need(40, 50, 256, op(), op()) == 0
    assert need(40, 50, 250, op(ld=250), op()) == 40 * 256                  # 40 lines of 256 bytes
    assert need(40, 50, 250, op(), op(data=4097)) == 50 * 256
    assert need(40, 50, 250, op(ld=250), op(ld=251)) == 40 * 256 + 50 * 256
    assert need(1, 50, 250, op(ld=250), op()) == 0                          # one line needs no leading dimension
    assert need(0, 50, 250, op(ld=250), op()) == 0


def test_torch_forms_refuse():
    import torch
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError):
        mpg.fp8_quantize(x)                                   # not on a CUDA device
    with pytest.raises(ValueError):
        mpg.fp8_quantize(x, fmt="e3m4")
    with pytest.raises(ValueError):
        mpg.fp8_quantize(x, block="column")
    with pytest.raises(ValueError):
        mpg.fp8_quantize(x[0])
    with pytest.raises(TypeError):
        mpg.fp8_quantize(x.double())
    a = torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        mpg.gemm_fp8(a, s, a, s)


def test_plain_quantizer_on_known_values():
    x = np.zeros((2, 256))
    x[0, 0], x[0, 1], x[0, 2] = 448.0, 17.0, -19.0            # 17, 19: halfway between 16, 18 and 20: ties to even
    x[0, 130] = 449.0                                         # needs the next power of two
    x[1, 3] = np.inf
    x[1, 4] = 2.0 ** -140
    qv, s = quantize(x, "e4m3", 1)
    assert s.tolist() == [[1.0, 2.0], [2.0 ** -126, 1.0]]
    assert qv[0, :3].tolist() == [448.0, 16.0, -20.0] and qv[0, 130] == 224.0
    assert np.isnan(qv[1, 3]) and qv[1, 4] == 0.0
    qv, s = quantize(np.full((3, 5), 57344.0 * 4), "e5m2", 128)
    assert s.tolist() == [[4.0]] and (widen(qv, s, 128) == 57344.0 * 4).all()
