"""The gated feed-forward product and its gradients, ``mpg_gated_gemm`` and
``mpg_gated_gemm_backward``, on torch tensors (argument marshalling only)."""
from __future__ import annotations

import ctypes

import mixed_precision_matmul_gb300 as _m

from .fp8 import _calls, _device_index, _on_device, _on_stream, _raw_stream, _types, _workspace

ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2
ACT_NAMES = {"silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}


class GatedLayer(ctypes.Structure):
    """mpg_gated_layer."""
    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("inner", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("x", ctypes.c_void_p),
        ("wg", ctypes.c_void_p),
        ("wu", ctypes.c_void_p),
        ("ldx", ctypes.c_int64),
        ("ldwg", ctypes.c_int64),
        ("ldwu", ctypes.c_int64),
    ]


def _declare(L):
    i64, i32, vp, sz, p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(GatedLayer)
    for f in (L.mpg_gated_gemm_workspace_size, L.mpg_gated_gemm_backward_workspace_size):
        f.argtypes, f.restype = [p], sz
    L.mpg_gated_gemm.argtypes, L.mpg_gated_gemm.restype = [p] + [vp, i64] * 3 + [vp, sz, vp], i32
    L.mpg_gated_gemm_backward.argtypes, L.mpg_gated_gemm_backward.restype = [p] + [vp, i64] * 6 + [vp, sz, vp], i32


def gated_gemm_raw(layer, Y, ldy, A=0, lda=0, B=0, ldb=0, workspace=0, workspace_bytes=0, stream=0,
                   check: bool = True) -> int:
    """mpg_gated_gemm with a :class:`GatedLayer` and device addresses."""
    st = _m.lib().mpg_gated_gemm(ctypes.byref(layer) if layer is not None else None, Y or None, ldy, A or None, lda,
                                 B or None, ldb, workspace or None, workspace_bytes, stream or None)
    if check and st:
        _m._check(st)
    return st


def gated_gemm_backward_raw(layer, dY, lddy, A, lda, B, ldb, dX, lddx, dWg, lddwg, dWu, lddwu, workspace=0,
                            workspace_bytes=0, stream=0, check: bool = True) -> int:
    """mpg_gated_gemm_backward with a :class:`GatedLayer` and device addresses."""
    st = _m.lib().mpg_gated_gemm_backward(ctypes.byref(layer) if layer is not None else None, dY or None, lddy, A or None,
                                          lda, B or None, ldb, dX or None, lddx, dWg or None, lddwg, dWu or None, lddwu,
                                          workspace or None, workspace_bytes, stream or None)
    if check and st:
        _m._check(st)
    return st


def _matrix(t, name, dtype=None, shape=None):
    """Leading dimension of a 16-bit matrix (of one type, or fp16 or bf16) with unit column stride."""
    torch = _types()[0]
    if t.dim() != 2:
        raise ValueError(f"{name} is a 2-D tensor")
    if dtype is None and t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    rows, cols = t.shape
    if rows and cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if rows < 2:
        return max(cols, 1)
    if t.stride(0) < cols:
        raise ValueError(f"the rows of {name} overlap")
    return max(t.stride(0), 1)


def _act(act):
    code = ACT_NAMES.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}")
    return code


def _kept_dtype(dtype):
    """Of what a layer keeps for its gradients: fp16, or the codes of mpg_gated_gemm in a bf16 layer."""
    torch = _types()[0]
    return torch.int16 if dtype == torch.bfloat16 else dtype


def _layer(x, wg, wu, act):
    _, _, _, codes = _types()
    ldx = _matrix(x, "x")
    if wg.dim() != 2 or x.shape[1] != wg.shape[1]:
        raise ValueError("x and wg have different hidden sizes")
    ldwg = _matrix(wg, "wg", x.dtype)
    ldwu = _matrix(wu, "wu", x.dtype, wg.shape)
    return GatedLayer(x.shape[0], x.shape[1], wg.shape[0], codes[x.dtype], act, x.data_ptr(), wg.data_ptr(), wu.data_ptr(),
                      ldx, ldwg, ldwu)


def _scratch(size, layer, workspace, device):
    """(workspace, address, bytes): the caller's, or one of the size that the call needs."""
    if workspace is None:
        need = int(size(ctypes.byref(layer)))
        workspace = _types()[0].empty(need, dtype=_types()[0].uint8, device=device)
    return (workspace, *_workspace(workspace))


def gated_gemm(x, wg, wu, act: str = "silu", keep: bool = False, workspace=None, stream=None):
    """``act(x @ wg.T) * (x @ wu.T)`` for 16-bit x (tokens, hidden) and wg and wu
    (inner, hidden), in one kernel.

    ``act`` is "silu", "gelu" or "gelu_tanh".  With ``keep`` returns ``(y, a, b)``,
    where a and b are what :func:`gated_gemm_backward` makes gradients from, act(g)
    and u act'(g) of the projections g and u: fp16 in an fp16 layer, and in a bf16
    layer int16 codes of a 16-bit type with more precision than bf16 (mpgemm.h says
    which) and less range: what is kept is infinite from 65504 on in fp16 and from 2^32
    on in a bf16 layer, and loses bits below 2^-14 and 2^-30.  Gradients are then
    infinite or NaN that are finite when the projections are computed again
    (``kept=None``).
    """
    torch = _types()[0]
    if stream is not None:
        return _on_stream(stream, [x, wg, wu, workspace], lambda: gated_gemm(x, wg, wu, act, keep, workspace))
    code = _act(act)
    if workspace is None:
        calls = _calls()
        r = calls.gated_gemm(x, wg, wu, code, keep) if calls else None
        if r is not None:
            if r.__class__ is int:
                _m._check(r)
            return r
    index = _device_index(x, wg, wu, workspace)
    if index != torch.cuda.current_device():
        return _on_device(index, lambda: gated_gemm(x, wg, wu, act, keep, workspace))
    layer = _layer(x, wg, wu, code)
    kept = _kept_dtype(x.dtype)
    outs = [torch.empty((layer.tokens, layer.inner), dtype=d, device=x.device)
            for d in ((x.dtype, kept, kept) if keep else (x.dtype,))]
    args = [v for t in outs for v in (t.data_ptr(), max(layer.inner, 1))] + [0, 0] * (3 - len(outs))
    _hold, *ws = _scratch(_m.lib().mpg_gated_gemm_workspace_size, layer, workspace, x.device)
    gated_gemm_raw(layer, *args, *ws, _raw_stream()(index))
    return tuple(outs) if keep else outs[0]


def gated_gemm_backward(dy, x, wg, wu, act: str = "silu", kept=None, need_dx: bool = True, need_dw: bool = True,
                        workspace=None, stream=None):
    """Gradients ``(dx, dwg, dwu)`` of :func:`gated_gemm` for dy (tokens, inner).

    ``kept`` is the ``(a, b)`` of ``gated_gemm(..., keep=True)``, whose range is
    smaller than the layer's; without it the projections are computed again, over the
    whole range.  What is not needed is None.
    """
    torch = _types()[0]
    a, b = kept if kept is not None else (None, None)
    if stream is not None:
        return _on_stream(stream, [dy, x, wg, wu, a, b, workspace],
                          lambda: gated_gemm_backward(dy, x, wg, wu, act, kept, need_dx, need_dw, workspace))
    code = _act(act)
    if workspace is None:
        calls = _calls()
        r = calls.gated_gemm_backward(dy, x, wg, wu, code, a, b, need_dx, need_dw) if calls else None
        if r is not None:
            if r.__class__ is int:
                _m._check(r)
            return r
    index = _device_index(dy, x, wg, wu, a, b, workspace)
    if index != torch.cuda.current_device():
        return _on_device(index, lambda: gated_gemm_backward(dy, x, wg, wu, act, kept, need_dx, need_dw, workspace))
    layer = _layer(x, wg, wu, code)
    shape = (layer.tokens, layer.inner)
    args = [dy.data_ptr(), _matrix(dy, "dy", x.dtype, shape)]
    for t, name in ((a, "a"), (b, "b")):
        if (t is None) != (kept is None):
            raise ValueError("a and b are kept together")
        args += [0, 0] if t is None else [t.data_ptr(), _matrix(t, name, _kept_dtype(x.dtype), shape)]
    # (a weight whose lines have gaps gets a gradient without them)
    outs = [torch.empty(t.shape, dtype=x.dtype, device=x.device) if need else None
            for t, need in ((x, need_dx), (wg, need_dw), (wu, need_dw))]
    for t in outs:
        args += [0, 0] if t is None else [t.data_ptr(), max(layer.hidden, 1)]
    _hold, *ws = _scratch(_m.lib().mpg_gated_gemm_backward_workspace_size, layer, workspace, x.device)
    gated_gemm_backward_raw(layer, *args, *ws, _raw_stream()(index))
    return tuple(outs)
