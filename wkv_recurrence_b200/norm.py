"""Binding of the RMS norm (wkv_rms_norm_* of include/wkv.h): the norm of the
residual stream, by groups (heads) of a row, in 16 or 32 bits or in e4m3 with
scales, and its gradients.

    s = x + residual (held in the residual's dtype),
    y = s / sqrt(mean over the group of s^2 + eps) * weight

Argument marshalling only, like api.py: every step runs in the library's
kernels, on the current stream of the inputs' device.
"""
from __future__ import annotations

import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from .api import _DT
from .gated import _call, _ptr, _tensor


def _rows(t: torch.Tensor, name: str):
    """(rows, row stride in elements) of [..., C] seen as [rows, C] without a copy."""
    C = t.shape[-1]
    if t.is_contiguous() or t.numel() == 0:
        return (t.numel() // C if C else math.prod(t.shape[:-1])), C
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    try:
        v = t.view(-1, C)
    except RuntimeError:
        raise ValueError(f"the leading axes of {name} must be seen as rows of one stride") from None
    return v.shape[0], v.stride(0)


def _value(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DT:
        raise TypeError(f"{name}: dtype {t.dtype} is not supported (float32 or bfloat16)")
    return _DT[t.dtype]


def _same(t, name: str, like: torch.Tensor) -> int:
    code = _value(t, name)
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}, the device of the other arguments")
    if t.shape != like.shape:
        raise ValueError(f"{name} must be {list(like.shape)}")
    return code


def _checked(x, weight, residual, eps: float, groups: int):
    """What forward and quantisation check alike: the library call's first arguments, and the residual's new tensor."""
    xc = _value(x, "x")
    if x.dim() < 1:
        raise ValueError("x must be [..., C]")
    C = x.shape[-1]
    if not eps > 0 or not math.isfinite(eps):
        raise ValueError("eps must be positive and finite")
    if groups < 1 or C % groups:
        raise ValueError("groups must divide the columns")
    _tensor(weight, "weight", x.device, (C,), torch.float32)
    N, xs = _rows(x, "x")
    if residual is None:
        return (N, C, groups, eps, x.data_ptr(), xc, xs, 0, xc, 0, weight.data_ptr())
    rc = _same(residual, "residual", x)
    if x.dtype == torch.float32 and residual.dtype != torch.float32:
        raise TypeError("residual must be float32 beside a float32 x")
    rs = _rows(residual, "residual")[1]
    return (N, C, groups, eps, x.data_ptr(), xc, xs, residual.data_ptr(), rc, rs, weight.data_ptr())


def _sum_out(x, residual, residual_out):
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without a residual")
        return None
    if residual_out is None:
        return torch.empty(x.shape, dtype=residual.dtype, device=x.device)
    _tensor(residual_out, "residual_out", x.device, x.shape, residual.dtype)
    return residual_out


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
    args = _checked(x, weight, residual, eps, groups)
    out_dtype = out_dtype or (x.dtype if out is None else out.dtype)
    if out_dtype not in _DT or (x.dtype == torch.float32 and out_dtype != torch.float32):
        raise TypeError(f"output dtype {out_dtype} is not supported for {x.dtype} inputs")
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    else:
        _tensor(out, "out", x.device, x.shape, out_dtype)
    s = _sum_out(x, residual, residual_out)
    _call(x.device, _abi.lib().wkv_rms_norm, "wkv_rms_norm", *args, out.data_ptr(), _DT[out_dtype], _ptr(s))
    return out, s


def rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                   groups: int = 1, block: int = 0, residual_out: Optional[torch.Tensor] = None):
    """``rms_norm`` with its output in 8 bits: (q, scale, s) with q [..., C]
    float8_e4m3fn, scale float32 [..., C / block] and q * scale close to y.
    block: columns per scale: 32, 64 or 128 (dividing C), or 0 for the whole
    row. scale = max |y| / 448 of its block, 1 for a block of zeros.
    """
    args = _checked(x, weight, residual, eps, groups)
    C = x.shape[-1]
    if block not in (0, 32, 64, 128) or (block and C % block):
        raise ValueError("block must be 0 (a whole row), or 32, 64 or 128 and divide the columns")
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    blocks = C // block if block else 1
    scale = torch.empty(x.shape[:-1] + (blocks,), dtype=torch.float32, device=x.device)
    s = _sum_out(x, residual, residual_out)
    _call(x.device, _abi.lib().wkv_rms_norm_quant, "wkv_rms_norm_quant", *args, q.data_ptr(), scale.data_ptr(), block,
          _ptr(s))
    return q, scale, s


def rms_norm_backward(gy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, gs: Optional[torch.Tensor] = None, *,
                      eps: float = 1e-6, groups: int = 1, workspace: Optional[torch.Tensor] = None):
    """Gradients of a loss with dL/dy = gy [..., C] and, from the stream's other
    reader, dL/ds = gs (s's dtype, or None): (ds, dweight). ds, in s's dtype, is
    the gradient of x and of the residual alike; dweight float32 [C] is summed
    over the rows. s: as ``rms_norm`` returned it (x itself without a residual).
    """
    sc = _value(s, "s")
    gc = _same(gy, "gy", s)
    if gy.dtype == torch.float32 and s.dtype != torch.float32:
        raise TypeError("s must be float32 beside a float32 gy")
    if s.dim() < 1:
        raise ValueError("s must be [..., C]")
    C, dev = s.shape[-1], s.device
    if not eps > 0 or not math.isfinite(eps):
        raise ValueError("eps must be positive and finite")
    if groups < 1 or C % groups:
        raise ValueError("groups must divide the columns")
    _tensor(weight, "weight", dev, (C,), torch.float32)
    _tensor(gy, "gy", dev, s.shape, gy.dtype)
    if gs is not None:
        _tensor(gs, "gs", dev, s.shape, s.dtype)
    N, ss = _rows(s, "s")
    need = _abi.lib().wkv_rms_norm_backward_workspace_size(N, C, groups)
    if need == 0:
        raise ValueError("invalid sizes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    ds = torch.empty(s.shape, dtype=s.dtype, device=dev)
    dw = torch.empty(C, dtype=torch.float32, device=dev)
    _call(dev, _abi.lib().wkv_rms_norm_backward, "wkv_rms_norm_backward", N, C, groups, eps, gy.data_ptr(), gc,
          s.data_ptr(), sc, ss, weight.data_ptr(), _ptr(gs), ds.data_ptr(), dw.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return ds, dw


class RMSNorm(torch.autograd.Function):
    """``rms_norm`` as a torch autograd function, differentiable in x, weight and
    residual: ``RMSNorm.apply(x, weight, residual, eps, groups)`` returns (y, s),
    or y alone where residual is None."""

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
