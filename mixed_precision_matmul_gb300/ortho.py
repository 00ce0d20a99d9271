"""The orthogonalised update, ``mpg_orthogonalize``, on torch tensors (argument
marshalling only)."""
from __future__ import annotations

import ctypes

import mixed_precision_matmul_gb300 as _m

from .fp8 import _device_index, _on_device, _on_stream, _raw_stream, _types, _workspace

#: a, b, c of the quintic step whose five applications bring singular values to 0.7 .. 1.2
NS_COEFFS = (3.4445, -4.7750, 2.0315)


def orthogonalize_workspace_size(m, n, batch=1) -> int:
    return int(_m.lib().mpg_orthogonalize_workspace_size(m, n, batch))


def orthogonalize_raw(m, n, batch, G, ldg, strideG, g_dtype, O, ldo, strideO, o_dtype, steps=5, coeffs=NS_COEFFS,
                      eps=1e-7, alpha=1.0, beta=0.0, workspace=0, workspace_bytes=0, stream=0,
                      check: bool = True) -> int:
    """mpg_orthogonalize on device addresses."""
    c = (ctypes.c_float * 3)(*coeffs) if coeffs is not None else None
    st = _m.lib().mpg_orthogonalize(m, n, batch, G or None, ldg, strideG, g_dtype, O or None, ldo, strideO, o_dtype,
                                    steps, c, eps, alpha, beta, workspace or None, workspace_bytes, stream or None)
    if check and st:
        _m._check(st)
    return st


def _lines(t, name):
    """(leading dimension, batch stride) of a (batch, m, n) tensor."""
    b, m, n = t.shape
    if t.numel() and n > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    ld = t.stride(1) if m > 1 else max(n, 1)
    if t.numel() and ld < n:
        raise ValueError(f"the rows of {name} overlap")
    return max(ld, 1), t.stride(0) if b > 1 else 0


def orthogonalize(G, O=None, steps: int = 5, coeffs=NS_COEFFS, eps: float = 1e-7, alpha: float = 1.0,
                  beta: float = 0.0, out_dtype=None, workspace=None, stream=None):
    """O = alpha * NS(G) + beta * O: the Newton-Schulz orthogonalisation of a
    matrix (m, n), or of each of a batch (batch, m, n), as the Muon optimiser
    takes of a momentum.

    G is fp32, fp16 or bf16 with unit column stride.  O is allocated with
    ``out_dtype`` (default bf16) when not given; with O given, ``alpha`` and
    ``beta`` fold the update into it, e.g. ``orthogonalize(M, O=W, alpha=-lr,
    beta=1 - lr * decay)``.  Returns O.
    """
    torch, _, _, codes = _types()
    if stream is not None:
        return _on_stream(stream, [G, O, workspace],
                          lambda: orthogonalize(G, O, steps, coeffs, eps, alpha, beta, out_dtype, workspace))
    if G.dim() not in (2, 3):
        raise ValueError("G is a matrix or a batch of matrices")
    if G.dtype not in codes:
        raise TypeError(f"unsupported dtype {G.dtype}")
    if len(coeffs) != 3:
        raise ValueError("three coefficients are expected")
    index = _device_index(G, O, workspace)
    if index != torch.cuda.current_device():
        return _on_device(index,
                          lambda: orthogonalize(G, O, steps, coeffs, eps, alpha, beta, out_dtype, workspace))
    if O is None:
        if beta != 0.0:
            raise ValueError("beta needs O")
        O = torch.empty(G.shape, dtype=out_dtype or torch.bfloat16, device=G.device)
    elif out_dtype is not None and O.dtype != out_dtype:
        raise ValueError("O has another dtype than out_dtype")
    if O.shape != G.shape:
        raise ValueError("shape mismatch")
    if O.dtype not in codes:
        raise TypeError(f"unsupported dtype {O.dtype}")
    g3, o3 = (G, O) if G.dim() == 3 else (G.unsqueeze(0), O.unsqueeze(0))
    batch, m, n = g3.shape
    if g3.numel() == 0:
        return O
    ldg, sg = _lines(g3, "G")
    ldo, so = _lines(o3, "O")
    if batch > 1 and so == 0:
        raise ValueError("the matrices of O overlap")
    if batch > 1 and sg == 0:
        # one matrix shared by the whole batch: the ABI's 0 means packed
        g3 = g3.contiguous()
        ldg, sg = _lines(g3, "G")
    if workspace is None:
        workspace = torch.empty(orthogonalize_workspace_size(m, n, batch), dtype=torch.uint8, device=G.device)
    orthogonalize_raw(m, n, batch, g3.data_ptr(), ldg, sg, codes[G.dtype], o3.data_ptr(), ldo, so, codes[O.dtype],
                      steps, coeffs, eps, alpha, beta, *_workspace(workspace), _raw_stream()(index))
    return O
