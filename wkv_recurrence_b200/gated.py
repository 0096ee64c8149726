"""Binding of the gated linear recurrence (wkv_gated_* of include/wkv.h).

Per channel, with a gate z for every token:

    h_t = f_t h_{t-1} + i_t x_t      gate "sigmoid": f = sigmoid(z), i = 1 - f
                                     gate "decay":   f = e^{-z},     i = 1

Every step runs in the library's kernels, on the current stream of the inputs'
device; the checks, allocations and the call itself are native
(csrc/wkv_torch.cpp).
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from ._native import ext
from .api import query_status


def gated_workspace_size(B: int, T: int, C: int) -> int:
    """Bytes of workspace ``gated_forward`` and ``gated_backward`` need for this shape (host-only)."""
    n = _abi.lib().wkv_gated_workspace_size(int(B), int(T), int(C))
    if n == 0:
        raise ValueError("invalid sizes")
    return int(n)


def gated_status(device=None) -> int:
    """Synchronise the current stream of ``device`` (default: the current one)
    and return and clear the status of the workspace that is kept for it: 0, or 6
    (WKV_ERR_WAIT_TIMEOUT) if a wait inside a ``gated_forward``,
    ``gated_backward`` or ``Gated`` on that stream, without a workspace of the
    caller's, gave up since the last query. The results of such a call are not
    valid. ``query_status`` is the same for a caller's workspace."""
    with torch.cuda.device(torch.cuda.current_device() if device is None else torch.device(device)):
        kept = ext().gated_kept_workspace(torch.cuda.current_device())
        return 0 if kept is None else query_status(kept)


def gated_checkpoints(x: torch.Tensor) -> torch.Tensor:
    """A tensor for the ``checkpoints`` of ``gated_forward`` over x [B, T, C]: the
    state in front of every 128 tokens, float32 [B, ceil(T / 128), C]."""
    return ext().gated_checkpoints(x)


def gated_forward(x: torch.Tensor, z: torch.Tensor, state: Optional[torch.Tensor] = None, *, gate: str = "sigmoid",
                  out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                  state_out: Optional[torch.Tensor] = None, checkpoints: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None):
    """The gated linear recurrence over a sequence: x, z [B, T, C] (float32 or
    bfloat16; z may be float32 beside a bfloat16 x), channel axis contiguous,
    any other strides. state: float32 [B, C], or None for zero. gate: "sigmoid"
    (z = -inf starts a sequence of its own) or "decay" (z as ``forward``'s w_t).

    Returns (out [B, T, C], state after the last token). state_out may be
    ``state``. checkpoints: a ``gated_checkpoints(x)`` tensor to be filled for
    ``gated_backward``. workspace: ``gated_workspace_size`` bytes, zero-filled
    once, for this operator alone; by default one is kept per stream (see
    ``gated_status``). A call that is captured into a graph gets one in the
    graph's memory, whose status cannot be queried: pass one where it matters.
    """
    return ext().gated_forward(x, z, state, gate, out_dtype, out, state_out, checkpoints, workspace)


def gated_backward(x: torch.Tensor, z: torch.Tensor, gout: torch.Tensor, state: Optional[torch.Tensor] = None,
                   dstate: Optional[torch.Tensor] = None, *, gate: str = "sigmoid",
                   checkpoints: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of a loss with dL/d out = gout [B, T, C] (contiguous, of the
    output's dtype) and dL/d (state after the last token) = dstate [B, C] (None:
    zero), for the x, z and state of a ``gated_forward``.

    Returns (dx, dz, dstate_in): contiguous, in the dtypes of x and z, and
    float32 [B, C]. checkpoints: as that forward filled them; None computes
    them again first (one more pass over x and z).
    """
    return ext().gated_backward(x, z, gout, state, dstate, gate, checkpoints, workspace)


def gated_step(state: torch.Tensor, x: torch.Tensor, z: torch.Tensor, *, gate: str = "sigmoid",
               out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               state_out: Optional[torch.Tensor] = None, inplace: bool = False):
    """One token for S streams: x, z [S, C] (channel axis contiguous), state
    float32 [S, C]. Returns (out [S, C], new state). With ``inplace=True`` the
    state tensor is updated in place and returned, as with state_out=state."""
    return ext().gated_step(state, x, z, gate, out_dtype, out, state_out, inplace)


class Gated(torch.autograd.Function):
    """The gated linear recurrence as a torch autograd function:
    ``Gated.apply(x, z, state, gate)`` returns (out, state after the last
    token), differentiable in x, z and state (which may be None). Under graph
    capture call ``gated_forward`` and ``gated_backward`` themselves."""

    @staticmethod
    def forward(ctx, x, z, state=None, gate="sigmoid"):
        marks = gated_checkpoints(x) if x.dim() == 3 and x.shape[1] > _abi.WKV_GATED_TILE else None
        out, state_out = gated_forward(x, z, state, gate=gate, checkpoints=marks)
        ctx.save_for_backward(x, z, state, marks)
        ctx.gate = gate
        ctx.set_materialize_grads(False)
        return out, state_out

    @staticmethod
    @once_differentiable
    def backward(ctx, gout, dstate):
        x, z, state, marks = ctx.saved_tensors
        gout = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if gout is None else gout.contiguous()
        dstate = None if dstate is None else dstate.contiguous()
        dx, dz, dstate_in = gated_backward(x, z, gout, state, dstate, gate=ctx.gate, checkpoints=marks)
        return dx, dz, None if state is None else dstate_in, None
