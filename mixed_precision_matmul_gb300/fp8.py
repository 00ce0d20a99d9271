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
def _calls():
    """The extension that makes the plain calls (csrc/torch_calls.cpp), or None
    where there is none for this torch and Python: every call then takes the
    Python form below, which costs the host 9 us more."""
    import importlib.machinery
    import importlib.util
    import warnings

    _types()                                    # torch first: the extension links to it
    lib = _m.lib()
    path = _m._build.torch_calls_path()
    loader = importlib.machinery.ExtensionFileLoader("_torch_calls", path)
    spec = importlib.util.spec_from_file_location("_torch_calls", path, loader=loader)
    try:
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"8-bit calls are marshalled in Python, build() makes the extension: {e}", RuntimeWarning)
        return None
    module.init(*(ctypes.cast(f, ctypes.c_void_p).value
                  for f in (lib.mpg_gemm_fp8, lib.mpg_gemm_fp8_workspace_size, lib.mpg_fp8_quantize)))
    return module


@functools.cache
def _default_options(c_dtype: int):
    return _m.options(c_dtype=c_dtype)


@functools.cache
def _raw_stream():
    """Handle of the current stream of a device index.  (torch.cuda.current_stream
    builds a Stream object first: 2 us a call of about 10.)"""
    torch = _types()[0]
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_stream(stream, tensors, call):
    """Run ``call()`` with ``stream`` current, so that what it allocates belongs
    to that stream, and keep ``tensors`` alive for the work enqueued there."""
    torch = _types()[0]
    _device_index(*tensors)
    if not isinstance(stream, torch.cuda.Stream):      # a handle, or any object that has one
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        stream = torch.cuda.ExternalStream(handle, device=tensors[0].device)
    with torch.cuda.stream(stream):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return call()


def _device_index(*tensors) -> int:
    """The CUDA device that all given tensors are on."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("operands are on different devices")
    if index < 0:
        raise ValueError("CUDA tensors expected")
    return index


def _workspace(workspace):
    """(address, bytes) of a given workspace, whose bytes have to be its own."""
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _on_device(index, call):
    """``call`` with device ``index`` current."""
    with _types()[0].cuda.device(index):
        return call()


def fp8_quantize_raw(rows, cols, X, ldx, x_dtype, fmt, scale_rows, Q, ldq, S, s_row, s_k, QT, ldqt, ST, st_row, st_k,
                     stream=0, check: bool = True) -> int:
    """mpg_fp8_quantize on device addresses (0 for a form that is not wanted)."""
    st = _m.lib().mpg_fp8_quantize(rows, cols, X or None, ldx, x_dtype, fmt, scale_rows, Q or None, ldq, S or None,
                                   s_row, s_k, QT or None, ldqt, ST or None, st_row, st_k, stream or None)
    if check and st:
        _m._check(st)
    return st


def _form(rows, cols, code, scale_rows, device):
    """(codes, their leading dimension, scales, row stride, k stride) of a rows x
    cols matrix: lines of codes start on 16-byte boundaries, and the scales of
    single rows lie block by block, which is how the product reads them
    fastest."""
    empty = _types()[0].empty_strided
    ld = (cols + 15) & ~15 or 1
    q = empty((rows, cols), (ld, 1), dtype=code, device=device)
    kb = (cols + BLOCK - 1) // BLOCK
    if scale_rows == 1:
        return q, ld, empty((rows, kb), (1, rows or 1), device=device, dtype=_types()[0].float32), 1, rows or 1
    sr = (rows + BLOCK - 1) // BLOCK
    return q, ld, empty((sr, kb), (kb or 1, 1), device=device, dtype=_types()[0].float32), kb or 1, 1


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
    code = dtypes.get(fmt)
    if code is None:
        raise ValueError(f"unknown 8-bit format {fmt!r}")
    scale_rows = 1 if block == "row" else BLOCK
    if scale_rows == BLOCK and block != "tile":
        raise ValueError("block is 'row' or 'tile'")
    calls = _calls()
    r = calls.quantize(x, fmt, scale_rows, transpose) if calls else None
    if r is not None:
        if r.__class__ is int:
            _m._check(r)
        return r
    if x.dim() != 2:
        raise ValueError("a 2-D tensor is expected")
    x_dtype = codes.get(x.dtype)
    if x_dtype is None:
        raise TypeError(f"unsupported dtype {x.dtype}")
    index = x.get_device()
    if index < 0:
        raise ValueError("CUDA tensors expected")
    if index != torch.cuda.current_device():
        return _on_device(index, lambda: fp8_quantize(x, fmt, block, transpose))
    rows, cols = x.shape
    ldx, unit = x.stride()
    if unit != 1 and rows and cols > 1:
        raise ValueError("x must be row-major with unit column stride")
    if rows < 2:
        ldx = cols or 1
    elif ldx < cols:
        raise ValueError("the rows of x overlap")
    device = x.device
    q, ldq, s, s_row, s_k = _form(rows, cols, code, scale_rows, device)
    if not transpose:
        if rows and cols:
            _m._check(_m.lib().mpg_fp8_quantize(rows, cols, x.data_ptr(), ldx, x_dtype, fmt, scale_rows, q.data_ptr(),
                                                ldq, s.data_ptr(), s_row, s_k, None, 0, None, 0, 0,
                                                _raw_stream()(index)))
        return q, s
    qt, ldqt, st, st_row, st_k = _form(cols, rows, code, scale_rows, device)
    if rows and cols:
        _m._check(_m.lib().mpg_fp8_quantize(rows, cols, x.data_ptr(), ldx, x_dtype, fmt, scale_rows, q.data_ptr(), ldq,
                                            s.data_ptr(), s_row, s_k, qt.data_ptr(), ldqt, st.data_ptr(), st_row, st_k,
                                            _raw_stream()(index)))
    return q, s, qt, st


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


def _operand(t, scale, name, index):
    """(description of an 8-bit tensor and its scales, rows, k)."""
    torch, formats, _, _ = _types()
    fmt = formats.get(t.dtype)
    if fmt is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if scale.dtype != torch.float32:
        raise TypeError(f"{name}: scales must be fp32")
    if t.get_device() != index or scale.get_device() != index:
        raise ValueError("operands are on different devices" if index >= 0 else "CUDA tensors expected")
    if t.dim() != 2 or scale.dim() != 2:
        raise ValueError(f"{name} and its scales are 2-D tensors")
    rows, k = t.shape
    ld, unit = t.stride()
    sr, sk = scale.shape
    s_row, s_k = scale.stride()
    kb = (k + BLOCK - 1) // BLOCK
    if sk == kb and sr == rows:
        scale_rows = 1
    elif sk == kb and sr == (rows + BLOCK - 1) // BLOCK:
        scale_rows = BLOCK
    else:
        raise ValueError(f"{name}: scales of shape {tuple(scale.shape)} fit neither 1 x 128 nor 128 x 128 blocks of "
                         f"{tuple(t.shape)}")
    if unit != 1 and k > 1 and rows:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if rows < 2:
        ld = k
    elif ld < k:
        raise ValueError(f"the rows of {name} overlap")
    return _m.Fp8Operand(t.data_ptr(), ld or 1, fmt, scale_rows, scale.data_ptr(), s_row, s_k), rows, k


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
    torch, _, _, codes = _types()
    if stream is not None:
        return _on_stream(stream, [A, a_scale, B, b_scale, C, workspace],
                          lambda: gemm_fp8(A, a_scale, B, b_scale, C, alpha, beta, out_dtype, workspace, opts))
    if C is None and opts is None and workspace is None and beta == 0.0:
        code = codes.get(out_dtype) if out_dtype is not None else _m.BF16
        calls = _calls()
        if calls and code is not None:
            r = calls.gemm_fp8(A, a_scale, B, b_scale, alpha, code)
            if r is not None:
                if r.__class__ is int:
                    _m._check(r)
                return r
    index = A.get_device()
    if index < 0:
        raise ValueError("CUDA tensors expected")
    if index != torch.cuda.current_device():
        return _on_device(index, lambda: gemm_fp8(A, a_scale, B, b_scale, C, alpha, beta, out_dtype, workspace, opts))
    a, m, k = _operand(A, a_scale, "A", index)
    b, n, kb = _operand(B, b_scale, "B", index)
    if kb != k:
        raise ValueError("A and B have different k")
    if C is None:
        if beta != 0.0:
            raise ValueError("beta needs C")
        C = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=A.device)
        ldc = n
    else:
        if C.get_device() != index:
            raise ValueError("operands are on different devices")
        if out_dtype is not None and C.dtype != out_dtype:
            raise ValueError("C has another dtype than out_dtype")
        if C.shape != (m, n):
            raise ValueError("shape mismatch")
        ldc, unit = C.stride()
        if m and n > 1 and unit != 1:
            raise ValueError("C must have unit column stride")
        if m < 2:
            ldc = n
        elif ldc < n:
            raise ValueError("the rows of C overlap")
    code = codes.get(C.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {C.dtype}")
    if m == 0 or n == 0:
        return C
    if opts is None:
        opts = _default_options(code)
    elif opts.c_dtype != code:
        o = _m.Options()
        ctypes.memmove(ctypes.byref(o), ctypes.byref(opts), ctypes.sizeof(_m.Options))
        o.c_dtype = code
        opts = o
    ws = ws_bytes = 0
    if workspace is None and (((a.data or 0) | (b.data or 0)) & 15 or (m > 1 and a.ld & 15) or (n > 1 and b.ld & 15)):
        # lines that TMA cannot describe are copied to aligned ones
        need = _m.lib().mpg_gemm_fp8_workspace_size(m, n, k, ctypes.byref(a), ctypes.byref(b))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=A.device)
    if workspace is not None:
        if workspace.get_device() != index:
            raise ValueError("operands are on different devices")
        ws, ws_bytes = _workspace(workspace)
    _m._check(_m.lib().mpg_gemm_fp8(m, n, k, a, b, C.data_ptr(), ldc, alpha, beta, ws, ws_bytes, _raw_stream()(index),
                                    opts))
    return C
