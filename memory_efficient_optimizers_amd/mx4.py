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


def _call(device: torch.device, fn, *args, what: str = "MX4 operators need tensors") -> None:
    """fn on the current stream of `device`, made current for the call if it is not."""
    if device.type != "cuda":
        raise ValueError(f"{what} on a GPU")
    if device.index == torch.cuda.current_device():
        fn(*args)
    else:
        with torch.cuda.device(device):
            fn(*args)


def _view(t: torch.Tensor, transposed: bool):
    """A matrix as the library takes it: row-major rows, `transposed` turned round for a
    column-major view (a row-major matrix's ``.t()``)."""
    if t.is_contiguous():
        return t, transposed
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
    cols, rows = x.shape if transposed else x.shape[::-1]
    if out is None:
        out = MX4Tensor.empty(rows, cols, x.device)
    elif out.shape != (rows, cols) or out.device != x.device:
        raise ValueError(f"out holds {out.shape} on {out.device}, expected {(rows, cols)} on {x.device}")
    v, tr = _view(x, transposed)
    if not v.is_contiguous() and v.numel() and ((v.shape[1] > 1 and v.stride(1) != 1) or
                                                (v.shape[0] > 1 and v.stride(0) < v.shape[1])):
        v = v.detach().contiguous()
    _call(x.device, _lib.meo_mx4_quantize, (v,), (out,), tr)
    return out


def mx4_dequantize(q: MX4Tensor, dtype: torch.dtype = torch.float32, transposed: bool = False,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of ``q`` [rows][cols], or of its transpose, in ``dtype`` (float32 or
    bfloat16; exact) or into ``out`` (a row- or column-major view)."""
    shape = q.shape[::-1] if transposed else q.shape
    if out is None:
        out = v = torch.empty(shape, dtype=dtype, device=q.device)
        tr = transposed
    elif out.shape != shape or out.device != q.device:
        raise ValueError(f"out of shape {tuple(out.shape)} on {out.device}, expected {shape} on {q.device}")
    else:
        v, tr = _view(out.detach(), transposed)
    _call(q.device, _lib.meo_mx4_dequantize, (v,), (q,), tr)
    return out


def mx4_matmul(a: MX4Tensor, b: MX4Tensor, dtype: torch.dtype = torch.float32,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``a`` [m][k] times the transpose of ``b`` [n][k]: [m][n] in ``dtype`` (float32 or
    bfloat16), summed in float32."""
    if out is None:
        out = torch.empty((a.codes.shape[0], b.codes.shape[0]), dtype=dtype, device=a.device)
    _call(a.device, _lib.meo_mx4_matmul, (a,), (b,), (out,))
    return out
