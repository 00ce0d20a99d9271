"""The norm of many gradients and their clipping, ``mpg_clip_grad_norm``, on
torch tensors (argument marshalling only)."""
from __future__ import annotations

import ctypes

import mixed_precision_matmul_gb300 as _m

from .fp8 import _calls, _device_index, _on_device, _on_stream, _raw_stream, _types, _workspace

#: what the norm is raised by in the factor max_norm / (norm + eps)
CLIP_EPS = 1e-6


class Grad(ctypes.Structure):
    """mpg_grad."""
    _fields_ = [
        ("g", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("count", ctypes.c_int64),
        ("g_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
    ]


def _declare(L):
    i64, i32, f32, vp, sz, p = (ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                                ctypes.POINTER(Grad))
    L.mpg_clip_grad_norm_workspace_size.argtypes, L.mpg_clip_grad_norm_workspace_size.restype = [i64, p], sz
    L.mpg_clip_grad_norm.argtypes, L.mpg_clip_grad_norm.restype = [i64, p, f32, f32, vp, vp, sz, vp], i32


def clip_grad_norm_raw(grads, max_norm, norm, eps=CLIP_EPS, workspace=0, workspace_bytes=0, stream=0,
                       check: bool = True) -> int:
    """mpg_clip_grad_norm with a list of :class:`Grad` and device addresses."""
    table = (Grad * len(grads))(*grads) if grads is not None else None
    st = _m.lib().mpg_clip_grad_norm(len(grads or ()), table, max_norm, eps, norm or None, workspace or None, workspace_bytes,
                                     stream or None)
    if check and st:
        _m._check(st)
    return st


def clip_grad_norm(grads, max_norm: float, out=None, eps: float = CLIP_EPS, workspace=None, stream=None):
    """The norm of all gradients together, an fp32 tensor on their device, and
    the gradients times ``min(1, max_norm / (norm + eps))``, in place or into the
    tensors of the list ``out``.

    ``grads`` is a list of fp32, fp16 and bf16 tensors of any shapes without gaps
    (their memory order may be any, and that of ``out`` the same).
    ``max_norm=float("inf")`` leaves the gradients as they are.
    """
    torch, _, _, codes = _types()
    grads = grads if isinstance(grads, (list, tuple)) else list(grads)
    outs = grads if out is None else out if isinstance(out, (list, tuple)) else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{len(outs)} results for {len(grads)} gradients")
    if not grads:
        raise ValueError("no gradients")
    if stream is not None:
        return _on_stream(stream, [*grads, *([] if outs is grads else outs), workspace],
                          lambda: clip_grad_norm(grads, max_norm, outs, eps, workspace))
    if workspace is None:
        calls = _calls()
        r = calls.clip_grad_norm(grads, outs, max_norm, eps) if calls else None
        if r is not None:
            if r.__class__ is int:
                _m._check(r)
            return r
    index = _device_index(*grads, *outs, workspace)
    if index != torch.cuda.current_device():
        return _on_device(index, lambda: clip_grad_norm(grads, max_norm, outs, eps, workspace))
    table = []
    for i, (g, o) in enumerate(zip(grads, outs)):
        for t in (g, o):
            if t.dtype not in codes:
                raise TypeError(f"gradient {i}: unsupported dtype {t.dtype}")
            if not _dense(t):
                raise ValueError(f"gradient {i} has gaps, or elements that share memory")
        if g.shape != o.shape:
            raise ValueError(f"gradient {i}: shape mismatch")
        if g.numel() and any(a != b for a, b, n in zip(g.stride(), o.stride(), g.shape) if n > 1):
            raise ValueError(f"gradient {i}: its result has another memory order")
        table.append(Grad(g.data_ptr(), o.data_ptr(), g.numel(), codes[g.dtype], codes[o.dtype]))
    norm = torch.empty((), dtype=torch.float32, device=grads[0].device)
    if workspace is None:
        need = int(_m.lib().mpg_clip_grad_norm_workspace_size(len(table), (Grad * len(table))(*table)))
        workspace = torch.empty(need, dtype=torch.uint8, device=norm.device)
    clip_grad_norm_raw(table, max_norm, norm.data_ptr(), eps, *_workspace(workspace), _raw_stream()(index))
    return norm


def _dense(t) -> bool:
    """Whether a tensor's elements fill a block of memory, each its own place."""
    if t.numel() == 0:
        return True
    expected = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if stride != expected:
            return False
        expected *= size
    return True
