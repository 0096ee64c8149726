"""Binding of the RMS norm (wkv_rms_norm_* of include/wkv.h): the norm of the
residual stream, by groups (heads) of a row, in 16 or 32 bits or in e4m3 with
scales, and its gradients.

    s = x + residual (held in the residual's dtype),
    y = s / sqrt(mean over the group of s^2 + eps) * weight

Every step runs in the library's kernels, on the current stream of the inputs'
device; the checks, allocations and the call itself are native
(csrc/wkv_torch.cpp).
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from ._native import ext


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
             groups: int = 1, out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None):
    """RMS norm of x + residual over the last axis, in ``groups`` equal parts
    (heads). x [..., C] float32 or bfloat16, rows of any one stride; weight [C]
    float32; residual of x's shape, float32 or of x's dtype, or None.

    Returns (y, s): y [..., C] in out_dtype (x's by default), s = x + residual
    in the residual's dtype (None without one). y is the norm of that s.
    residual_out may be ``residual`` where that is contiguous (in place).
    """
    return ext().rms_norm(x, weight, residual, eps, groups, out_dtype, out, residual_out)


def rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                   groups: int = 1, block: int = 0, residual_out: Optional[torch.Tensor] = None):
    """``rms_norm`` with its output in 8 bits: (q, scale, s) with q [..., C]
    float8_e4m3fn, scale float32 [..., C / block] and q * scale close to y.
    block: columns per scale: 32, 64 or 128 (dividing C), or 0 for the whole
    row. scale = max |y| / 448 of its block, 1 for a block of zeros. q is y / scale
    rounded to e4m3; next to the middle of two e4m3 numbers either may be taken.
    Columns whose y is NaN are NaN in q and left out of the maximum.
    """
    return ext().rms_norm_quant(x, weight, residual, eps, groups, block, residual_out)


def rms_norm_backward(gy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, gs: Optional[torch.Tensor] = None, *,
                      eps: float = 1e-6, groups: int = 1, workspace: Optional[torch.Tensor] = None):
    """Gradients of a loss with dL/dy = gy [..., C] and, from the stream's other
    reader, dL/ds = gs (s's dtype, or None): (ds, dweight). ds, in s's dtype, is
    the gradient of x and of the residual alike; dweight float32 [C] is summed
    over the rows. s: as ``rms_norm`` returned it (x itself without a residual).
    """
    return ext().rms_norm_backward(gy, s, weight, gs, eps, groups, workspace)


class RMSNorm(torch.autograd.Function):
    """``rms_norm`` as a torch autograd function, differentiable in x, weight and
    residual: ``RMSNorm.apply(x, weight, residual, eps, groups)`` returns (y, s),
    or y alone where residual is None. Under graph capture call ``rms_norm`` and
    ``rms_norm_backward`` themselves."""

    @staticmethod
    def forward(ctx, x, weight, residual=None, eps=1e-6, groups=1):
        y, s = rms_norm(x, weight, residual, eps=eps, groups=groups)
        ctx.save_for_backward(x if residual is None else s, weight)
        ctx.eps, ctx.groups, ctx.x_dtype = eps, groups, x.dtype
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        return (y, s) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gs=None):
        s, weight = ctx.saved_tensors
        gy = torch.zeros(s.shape, dtype=ctx.x_dtype, device=s.device) if gy is None else gy.contiguous()
        gs = None if gs is None else gs.contiguous()
        ds, dw = rms_norm_backward(gy, s, weight, gs, eps=ctx.eps, groups=ctx.groups)
        return ds.to(ctx.x_dtype), dw, ds if ctx.has_residual else None, None, None
