"""The cross entropy of a projection onto a vocabulary and its gradients,
``mpg_linear_cross_entropy`` and ``mpg_linear_cross_entropy_backward``, on torch
tensors (argument marshalling only)."""
from __future__ import annotations

import ctypes

import mixed_precision_matmul_gb300 as _m

from .fp8 import _calls, _device_index, _on_device, _on_stream, _raw_stream, _types
from .gated import _matrix, _scratch


class VocabLoss(ctypes.Structure):
    """mpg_vocab_loss."""
    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("x", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("ldx", ctypes.c_int64),
        ("ldw", ctypes.c_int64),
        ("target", ctypes.c_void_p),
        ("target_bytes", ctypes.c_int32),
        ("target_stride", ctypes.c_int64),
        ("ignore_index", ctypes.c_int64),
    ]


def _declare(L):
    i64, i32, vp, sz, p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(VocabLoss)
    for f in (L.mpg_linear_cross_entropy_workspace_size, L.mpg_linear_cross_entropy_backward_workspace_size):
        f.argtypes, f.restype = [p], sz
    L.mpg_linear_cross_entropy.argtypes, L.mpg_linear_cross_entropy.restype = [p, vp, vp, vp, sz, vp], i32
    L.mpg_linear_cross_entropy_backward.argtypes = [p, vp, vp, i64, vp, i64, vp, i64, vp, sz, vp]
    L.mpg_linear_cross_entropy_backward.restype = i32


def linear_cross_entropy_raw(desc, loss, lse, workspace=0, workspace_bytes=0, stream=0, check: bool = True) -> int:
    """mpg_linear_cross_entropy with a :class:`VocabLoss` and device addresses."""
    st = _m.lib().mpg_linear_cross_entropy(ctypes.byref(desc) if desc is not None else None, loss or None, lse or None,
                                           workspace or None, workspace_bytes, stream or None)
    if check and st:
        _m._check(st)
    return st


def linear_cross_entropy_backward_raw(desc, lse, dloss, dloss_stride, dX, lddx, dW, lddw, workspace=0, workspace_bytes=0,
                                      stream=0, check: bool = True) -> int:
    """mpg_linear_cross_entropy_backward with a :class:`VocabLoss` and device addresses."""
    st = _m.lib().mpg_linear_cross_entropy_backward(ctypes.byref(desc) if desc is not None else None, lse or None,
                                                    dloss or None, dloss_stride, dX or None, lddx, dW or None, lddw,
                                                    workspace or None, workspace_bytes, stream or None)
    if check and st:
        _m._check(st)
    return st


def _desc(x, w, target, ignore_index):
    torch, _, _, codes = _types()
    ldx = _matrix(x, "x")
    if w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x and w have different hidden sizes")
    ldw = _matrix(w, "w", x.dtype)
    if target.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"targets are int64 or int32, not {target.dtype}")
    if tuple(target.shape) != (x.shape[0],):
        raise ValueError(f"targets of shape {tuple(target.shape)} for {x.shape[0]} tokens")
    return VocabLoss(x.shape[0], x.shape[1], w.shape[0], codes[x.dtype], x.data_ptr(), w.data_ptr(), ldx, ldw,
                     target.data_ptr(), target.element_size(), target.stride(0), ignore_index)


def linear_cross_entropy(x, w, target, ignore_index: int = -100, workspace=None, stream=None):
    """``(loss, lse)`` of each token, fp32: the cross entropy of logits ``x @ w.T``
    with the classes ``target`` and the log of the sum of their exponentials,
    without keeping the logits.

    x is (tokens, hidden) and w (vocab, hidden), 16 bits; target int64 or int32
    (tokens,).  Both results are 0 where target is ``ignore_index``, and NaN where
    it is neither that nor a class.
    """
    torch = _types()[0]
    if stream is not None:
        return _on_stream(stream, [x, w, target, workspace], lambda: linear_cross_entropy(x, w, target, ignore_index, workspace))
    if workspace is None:
        calls = _calls()
        r = calls.linear_cross_entropy(x, w, target, ignore_index) if calls else None
        if r is not None:
            if r.__class__ is int:
                _m._check(r)
            return r
    index = _device_index(x, w, target, workspace)
    if index != torch.cuda.current_device():
        return _on_device(index, lambda: linear_cross_entropy(x, w, target, ignore_index, workspace))
    desc = _desc(x, w, target, ignore_index)
    loss, lse = (torch.empty(desc.tokens, dtype=torch.float32, device=x.device) for _ in range(2))
    _hold, *ws = _scratch(_m.lib().mpg_linear_cross_entropy_workspace_size, desc, workspace, x.device)
    linear_cross_entropy_raw(desc, loss.data_ptr(), lse.data_ptr(), *ws, _raw_stream()(index))
    return loss, lse


def linear_cross_entropy_backward(x, w, target, lse, dloss, ignore_index: int = -100, need_dx: bool = True,
                                  need_dw: bool = True, workspace=None, stream=None):
    """Gradients ``(dx, dw)`` of :func:`linear_cross_entropy`'s loss for ``dloss``
    (tokens,), fp32 (an expanded one too: ``(1 / count).expand(tokens)`` for the
    mean).  ``lse`` is the forward call's.  What is not needed is None.  Rows of x
    whose token is ignored are multiplied by 0: infinities and NaN there make dw NaN.
    """
    torch = _types()[0]
    if stream is not None:
        return _on_stream(stream, [x, w, target, lse, dloss, workspace],
                          lambda: linear_cross_entropy_backward(x, w, target, lse, dloss, ignore_index, need_dx, need_dw,
                                                                workspace))
    if workspace is None:
        calls = _calls()
        r = calls.linear_cross_entropy_backward(x, w, target, lse, dloss, ignore_index, need_dx, need_dw) if calls else None
        if r is not None:
            if r.__class__ is int:
                _m._check(r)
            return r
    index = _device_index(x, w, target, lse, dloss, workspace)
    if index != torch.cuda.current_device():
        return _on_device(index, lambda: linear_cross_entropy_backward(x, w, target, lse, dloss, ignore_index, need_dx,
                                                                       need_dw, workspace))
    desc = _desc(x, w, target, ignore_index)
    for t, name in ((lse, "lse"), (dloss, "dloss")):
        if t.dtype != torch.float32:
            raise TypeError(f"{name} is fp32, not {t.dtype}")
        if tuple(t.shape) != (desc.tokens,):
            raise ValueError(f"{name} of shape {tuple(t.shape)} for {desc.tokens} tokens")
    if desc.tokens > 1 and lse.stride(0) != 1:
        raise ValueError("lse must be contiguous")
    outs = [torch.empty(t.shape, dtype=x.dtype, device=x.device) if need else None for t, need in ((x, need_dx), (w, need_dw))]
    args = []
    for t in outs:
        args += [0, 0] if t is None else [t.data_ptr(), max(desc.hidden, 1)]
    _hold, *ws = _scratch(_m.lib().mpg_linear_cross_entropy_backward_workspace_size, desc, workspace, x.device)
    linear_cross_entropy_backward_raw(desc, lse.data_ptr(), dloss.data_ptr(), dloss.stride(0), *args, *ws, _raw_stream()(index))
    return tuple(outs)
