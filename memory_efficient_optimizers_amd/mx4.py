"""MX4 matrices (4-bit microscaled, MXFP4): quantize, read back, multiply.

A matrix is held as an ``MX4Tensor``: 4-bit codes and one power-of-two scale per 32
consecutive values of a row, 17/32 byte per value. The arithmetic runs in the library's
HIP kernels; the functions here allocate the outputs, take strided and transposed views
as they are, and run on the values' device and its current stream. They are not
differentiable. ``GaLoreAdamW`` holds its projector this way with
``projector_dtype=torch.float4_e2m1fn_x2``.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._lib import MX4Tensor

__all__ = ["MX4Tensor", "mx4_quantize", "mx4_dequantize", "mx4_matmul"]


def _on_gpu(*devices) -> None:
    for d in devices:
        if d.type != "cuda":
            raise ValueError("MX4 operators need tensors on a GPU")


def _view(t: torch.Tensor, transposed: bool):
    """A matrix as the library takes it: row-major rows, `transposed` turned round for a
    column-major view (a row-major matrix's ``.t()``)."""
    row_major = t.shape[1] <= 1 or (t.stride(1) == 1 and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]))
    if not row_major and (t.shape[0] <= 1 or (t.stride(0) == 1 and t.stride(1) >= t.shape[0])):
        return t.t(), not transposed
    return t, transposed


def mx4_quantize(x: torch.Tensor, transposed: bool = False, out: Optional[MX4Tensor] = None) -> MX4Tensor:
    """``x`` (2-D, float32 or bfloat16) in MX4, blocks along its rows; with ``transposed``
    the transpose of ``x``, blocks down its columns. A view whose rows and columns are
    both strided is copied first."""
    if x.dim() != 2:
        raise ValueError("mx4_quantize takes a matrix")
    _on_gpu(x.device)
    rows, cols = (x.shape[1], x.shape[0]) if transposed else x.shape
    if out is None:
        out = MX4Tensor.empty(rows, cols, x.device)
    elif out.shape != (rows, cols) or out.device != x.device:
        raise ValueError(f"out holds {out.shape} on {out.device}, expected {(rows, cols)} on {x.device}")
    v, tr = _view(x.detach(), transposed)
    if v.numel() and v.shape[1] > 1 and v.stride(1) != 1 or (v.shape[0] > 1 and v.stride(0) < v.shape[1]):
        v = v.contiguous()
    with torch.cuda.device(x.device):
        _lib.meo_mx4_quantize([v], [out], tr)
    return out


def mx4_dequantize(q: MX4Tensor, dtype: torch.dtype = torch.float32, transposed: bool = False,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of ``q`` [rows][cols], or of its transpose, in ``dtype`` (float32 or
    bfloat16; exact) or into ``out`` (a row- or column-major view)."""
    _on_gpu(q.device)
    shape = (q.shape[1], q.shape[0]) if transposed else q.shape
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
    elif tuple(out.shape) != tuple(shape) or out.device != q.device:
        raise ValueError(f"out of shape {tuple(out.shape)} on {out.device}, expected {shape} on {q.device}")
    v, tr = _view(out.detach(), transposed)
    with torch.cuda.device(q.device):
        _lib.meo_mx4_dequantize([v], [q], tr)
    return out


def mx4_matmul(a: MX4Tensor, b: MX4Tensor, dtype: torch.dtype = torch.float32,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``a`` [m][k] times the transpose of ``b`` [n][k]: [m][n] in ``dtype`` (float32 or
    bfloat16), summed in float32."""
    _on_gpu(a.device, b.device)
    if out is None:
        out = torch.empty((a.shape[0], b.shape[0]), dtype=dtype, device=a.device)
    with torch.cuda.device(a.device):
        _lib.meo_mx4_matmul([a], [b], [out.detach()])
    return out
