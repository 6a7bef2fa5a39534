"""Orthogonalization of matrices by Newton-Schulz steps, the direction of the Muon optimizer
(``Muon`` in ``optim.py`` takes its steps with it). The arithmetic runs in the library's HIP
kernels on the tensors' device and its current stream. Not differentiable.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Union

import torch

from . import _lib
from .mx4 import _call

__all__ = ["orthogonalize"]


def _row_major(t: torch.Tensor) -> bool:
    try:
        _lib._ns_row_stride(t, "")
    except ValueError:
        return False
    return True


def orthogonalize(x: Union[torch.Tensor, Sequence[torch.Tensor]], steps: int = 5,
                  coefficients=_lib.NS_COEFFICIENTS, eps: float = 1e-7,
                  out: Union[torch.Tensor, Sequence[torch.Tensor], None] = None
                  ) -> Union[torch.Tensor, List[torch.Tensor]]:
    """The matrices of ``x`` (its last two dims; float32 or bfloat16; leading dims a batch)
    after ``steps`` Newton-Schulz steps X <- a X + (b A + c A^2) X, A = X X^T, from
    X / max(norm, eps), in bfloat16: singular vectors stay, singular values come near 1.
    ``coefficients``: one (a, b, c), or one for each step.

    ``x`` may be a list, which is worked on together (many small matrices take little longer
    than one). Row-major and column-major views are taken as they are, others copied first;
    results are laid out as their ``x``. ``out``: where they go (bfloat16, ``x``'s shapes); it may
    be ``x`` itself, and must not overlap anything else."""
    single = isinstance(x, torch.Tensor)
    xs = [x] if single else list(x)
    outs: Sequence[Optional[torch.Tensor]] = [None] * len(xs) if out is None else [out] if single else list(out)
    if len(outs) != len(xs):
        raise ValueError("x and out differ in length")
    hp = _lib.orthogonalize_hparams(steps, coefficients, eps)
    if not xs:
        _lib.meo_orthogonalize_validate(hp, [], [])
        return []
    if any(t.device != xs[0].device for t in xs):
        raise ValueError("the matrices must be on one device")
    src, dst, res = [], [], []
    for t, o in zip(xs, outs):
        if t.dim() < 2:
            raise ValueError("orthogonalize takes matrices (two or more dims)")
        if t.requires_grad:
            t = t.detach()
        # the transpose's result is the result's transpose: either orientation is worked on as it lies
        if o is None and t.is_contiguous():
            v, o = t, torch.empty_like(t, dtype=torch.bfloat16, memory_format=torch.contiguous_format)
            d = o
        elif o is None:
            flip = not _row_major(t) and _row_major(t.mT)
            v = t.mT if flip else t
            v = v if flip or _row_major(v) else v.contiguous()
            d = torch.empty(v.shape, dtype=torch.bfloat16, device=v.device)
            o = d.mT if flip else d
        else:
            if o.shape != t.shape or o.device != t.device:
                raise ValueError(f"out of shape {tuple(o.shape)} on {o.device}, expected {tuple(t.shape)} on {t.device}")
            d = o.detach()
            flip = not _row_major(d)
            v, d = (t.mT, d.mT) if flip else (t, d)
            v = v if _row_major(v) else v.contiguous()
        src.append(v)
        dst.append(d)
        res.append(o)
    arr = _lib._ns_matrices(src, dst)
    size = _lib.meo_orthogonalize_workspace_size(hp, arr, dst)
    _call(xs[0].device, lambda: _lib.meo_orthogonalize(hp, arr, dst, _lib.workspace(size, xs[0].device)),
          what="orthogonalize needs matrices")
    return res[0] if single else res
