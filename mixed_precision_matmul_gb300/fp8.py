"""8-bit operands with a scale for each block of 128: ``mpg_fp8_quantize`` and
``mpg_gemm_fp8`` on torch tensors (argument marshalling only)."""
from __future__ import annotations

import ctypes
import functools

import mixed_precision_matmul_gb300 as _m

E4M3, E5M2 = 0, 1
FORMAT_NAMES = {"e4m3": E4M3, "e5m2": E5M2}
BLOCK = 128


@functools.cache
def _types():
    """(torch, {8-bit torch dtype: format}, {format: 8-bit torch dtype}, {dtype: mpg_dtype})."""
    import torch
    formats = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
    codes = {torch.float32: _m.F32, torch.float16: _m.F16, torch.bfloat16: _m.BF16}
    return torch, formats, {f: d for d, f in formats.items()}, codes


@functools.cache
def _default_options(c_dtype: int):
    return _m.options(c_dtype=c_dtype)


def _on_stream(stream, tensors, call):
    """Run ``call()`` with ``stream`` current, so that what it allocates belongs
    to that stream, and keep ``tensors`` alive for the work enqueued there."""
    torch = _types()[0]
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=tensors[0].device)
    with torch.cuda.stream(stream):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return call()


def _current(device):
    """Handle of the current stream of a tensor's device."""
    return _types()[0].cuda.current_stream(device).cuda_stream


def _check_device(*tensors):
    device = tensors[0].device
    if device.type != "cuda":
        raise ValueError("CUDA tensors expected")
    for t in tensors[1:]:
        if t is not None and t.device != device:
            raise ValueError("operands are on different devices")
    return device


def fp8_quantize_raw(rows, cols, X, ldx, x_dtype, fmt, scale_rows, Q, ldq, S, s_row, s_k, QT, ldqt, ST, st_row, st_k,
                     stream=0, check: bool = True) -> int:
    """mpg_fp8_quantize on device addresses (0 for a form that is not wanted)."""
    st = _m.lib().mpg_fp8_quantize(rows, cols, X or None, ldx, x_dtype, fmt, scale_rows, Q or None, ldq, S or None,
                                   s_row, s_k, QT or None, ldqt, ST or None, st_row, st_k, stream or None)
    if check and st:
        _m._check(st)
    return st


def _codes(rows, cols, dtype, device):
    """rows x cols 8-bit tensor whose lines start on 16-byte boundaries."""
    torch = _types()[0]
    ld = -(-cols // 16) * 16
    t = torch.empty((rows, ld), dtype=dtype, device=device)
    return t if ld == cols else t[:, :cols]


def _scales(rows, cols, scale_rows, device):
    """Scales of a rows x cols matrix; per-row scales lie block by block, which
    is how the product reads them fastest."""
    torch = _types()[0]
    kb = -(-cols // BLOCK)
    if scale_rows == 1:
        return torch.empty((kb, rows), dtype=torch.float32, device=device).t()
    return torch.empty((-(-rows // BLOCK), kb), dtype=torch.float32, device=device)


def fp8_quantize(x, fmt="e4m3", block: str = "row", transpose: bool = False, stream=None):
    """Quantise a 2-D CUDA tensor (fp32, fp16 or bf16, unit column stride) to 8
    bits with a power-of-two scale for each block of 128.

    ``block`` "row": blocks of 1 x 128 along each row; "tile": 128 x 128.
    Returns ``(q, s)``, or with ``transpose`` ``(q, s, qt, st)``, where ``qt`` is
    the transposed matrix with its blocks along the rows of ``x`` (what the
    gradient of the weights contracts over), made in the same pass.  ``q`` is a
    float8 tensor of x's shape, ``s`` fp32 of (rows or blocks of rows, blocks of
    128 columns); x is approximately ``q * s`` block by block.
    """
    torch, _, dtypes, codes = _types()
    if stream is not None:
        return _on_stream(stream, [x], lambda: fp8_quantize(x, fmt, block, transpose))
    fmt = FORMAT_NAMES.get(fmt, fmt)
    if fmt not in dtypes:
        raise ValueError(f"unknown 8-bit format {fmt!r}")
    if block not in ("row", "tile"):
        raise ValueError("block is 'row' or 'tile'")
    if x.dim() != 2:
        raise ValueError("a 2-D tensor is expected")
    if x.dtype not in codes:
        raise TypeError(f"unsupported dtype {x.dtype}")
    device = _check_device(x)
    rows, cols = x.shape
    if rows and cols > 1 and x.stride(1) != 1:
        raise ValueError("x must be row-major with unit column stride")
    ldx = x.stride(0) if rows > 1 else max(cols, 1)
    if ldx < cols:
        raise ValueError("the rows of x overlap")
    scale_rows = 1 if block == "row" else BLOCK
    q = _codes(rows, cols, dtypes[fmt], device)
    s = _scales(rows, cols, scale_rows, device)
    qt = st = None
    if transpose:
        qt = _codes(cols, rows, dtypes[fmt], device)
        st = _scales(cols, rows, scale_rows, device)
    if rows and cols:
        with torch.cuda.device(device):
            fp8_quantize_raw(rows, cols, x.data_ptr(), ldx, codes[x.dtype], fmt, scale_rows,
                             q.data_ptr(), q.stride(0), s.data_ptr(), s.stride(0), s.stride(1),
                             qt.data_ptr() if transpose else 0, qt.stride(0) if transpose else 0,
                             st.data_ptr() if transpose else 0, st.stride(0) if transpose else 0,
                             st.stride(1) if transpose else 0, _current(device))
    return (q, s, qt, st) if transpose else (q, s)


def gemm_fp8_raw(m, n, k, A, B, C, ldc, alpha, beta, workspace=0, workspace_bytes=0, stream=0, opts=None,
                 check: bool = True) -> int:
    """mpg_gemm_fp8 with :class:`Fp8Operand` descriptions and device addresses."""
    st = _m.lib().mpg_gemm_fp8(m, n, k, ctypes.byref(A) if A is not None else None,
                               ctypes.byref(B) if B is not None else None, C or None, ldc, alpha, beta,
                               workspace or None, workspace_bytes, stream or None,
                               ctypes.byref(opts) if opts is not None else None)
    if check and st:
        _m._check(st)
    return st


def _operand(t, scale, name, formats):
    """The description of an 8-bit tensor and its scales."""
    torch = _types()[0]
    if t.dim() != 2 or scale.dim() != 2:
        raise ValueError(f"{name} and its scales are 2-D tensors")
    fmt = formats.get(t.dtype)
    if fmt is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if scale.dtype != torch.float32:
        raise TypeError(f"{name}: scales must be fp32")
    rows, k = t.shape
    kb = -(-k // BLOCK)
    if tuple(scale.shape) == (rows, kb):
        scale_rows = 1
    elif tuple(scale.shape) == (-(-rows // BLOCK), kb):
        scale_rows = BLOCK
    else:
        raise ValueError(f"{name}: scales of shape {tuple(scale.shape)} fit neither 1 x 128 nor 128 x 128 blocks of "
                         f"{tuple(t.shape)}")
    if rows and k > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    ld = t.stride(0) if rows > 1 else max(k, 1)
    if rows and ld < k:
        raise ValueError(f"the rows of {name} overlap")
    return _m.Fp8Operand(t.data_ptr(), max(ld, k, 1), fmt, scale_rows, scale.data_ptr(), scale.stride(0),
                         scale.stride(1))


def gemm_fp8(A, a_scale, B, b_scale, C=None, alpha: float = 1.0, beta: float = 0.0, out_dtype=None, workspace=None,
             opts=None, stream=None):
    """C = alpha * A @ B.T + beta * C for 8-bit A (m, k) and B (n, k) with a
    scale for each block of 128 along k.

    A and B are float8_e4m3fn or float8_e5m2 with unit column stride; their
    scales are fp32 of shape (rows, ceil(k / 128)) or (ceil(rows / 128),
    ceil(k / 128)), any strides.  C is fp32, fp16 or bf16 (m, n) with unit
    column stride, allocated with ``out_dtype`` (default bf16) when not given.
    Returns C.  The forward product of a layer is ``gemm_fp8(xq, xs, wq, ws)``,
    the gradient of its input ``gemm_fp8(dyq, dys, wqt, wst)`` and that of its
    weights ``gemm_fp8(dyqt, dyst, xqt, xst)``.
    """
    torch, formats, _, codes = _types()
    if stream is not None:
        return _on_stream(stream, [A, a_scale, B, b_scale, C, workspace],
                          lambda: gemm_fp8(A, a_scale, B, b_scale, C, alpha, beta, out_dtype, workspace, opts))
    device = _check_device(A, a_scale, B, b_scale, C, workspace)
    a = _operand(A, a_scale, "A", formats)
    b = _operand(B, b_scale, "B", formats)
    m, k = A.shape
    n = B.shape[0]
    if B.shape[1] != k:
        raise ValueError("A and B have different k")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta needs C")
        C = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=device)
    elif out_dtype is not None and C.dtype != out_dtype:
        raise ValueError("C has another dtype than out_dtype")
    if tuple(C.shape) != (m, n):
        raise ValueError("shape mismatch")
    if C.dtype not in codes or (m and n > 1 and C.stride(1) != 1):
        raise ValueError("C must be fp32, fp16 or bf16 with unit column stride")
    ldc = C.stride(0) if m > 1 else max(n, 1)
    if m and ldc < n:
        raise ValueError("the rows of C overlap")
    if m == 0 or n == 0:
        return C
    code = codes[C.dtype]
    if opts is None:
        opts = _default_options(code)
    elif opts.c_dtype != code:
        o = _m.Options()
        ctypes.memmove(ctypes.byref(o), ctypes.byref(opts), ctypes.sizeof(_m.Options))
        o.c_dtype = code
        opts = o
    with torch.cuda.device(device):
        need = _m.lib().mpg_gemm_fp8_workspace_size(m, n, k, ctypes.byref(a), ctypes.byref(b))
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        gemm_fp8_raw(m, n, k, a, b, C.data_ptr(), ldc, alpha, beta,
                     workspace.data_ptr() if workspace is not None else 0,
                     workspace.numel() * workspace.element_size() if workspace is not None else 0, _current(device), opts)
    return C
