"""Binding of the gated linear recurrence (wkv_gated_* of include/wkv.h).

Per channel, with a gate z for every token:

    h_t = f_t h_{t-1} + i_t x_t      gate "sigmoid": f = sigmoid(z), i = 1 - f
                                     gate "decay":   f = e^{-z},     i = 1

Argument marshalling only, like api.py: every step runs in the library's
kernels, on the current stream of the inputs' device.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from .api import _DT

GATES = {"sigmoid": _abi.WKV_GATE_SIGMOID, "decay": _abi.WKV_GATE_DECAY}

_workspaces = {}


def _tensor(t, name: str, dev: torch.device, shape, dtype) -> None:
    """A contiguous CUDA tensor of this device, shape and type, or an error that says what is wrong."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, the device of the other arguments")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _inputs(x, z, dims: int, what: str, gate: str):
    """Checks x and z; their type codes and the gate's."""
    for t, name in ((x, "x"), (z, "z")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype not in _DT:
            raise TypeError(f"{name}: dtype {t.dtype} is not supported (float32 or bfloat16)")
    if x.dim() != dims or x.shape != z.shape:
        raise ValueError(f"x and z must both be {what}")
    if x.device != z.device:
        raise ValueError("x and z must be on one device")
    if x.shape[-1] > 1 and (x.stride(-1) != 1 or z.stride(-1) != 1):
        raise ValueError("the channel axis of x and z must be contiguous")
    if z.dtype != x.dtype and z.dtype != torch.float32:
        raise TypeError("z must be float32 or of x's dtype")
    if gate not in GATES:
        raise ValueError(f"gate must be one of {sorted(GATES)}")
    return _DT[x.dtype], _DT[z.dtype], GATES[gate]


def _out_code(x, out_dtype) -> int:
    if out_dtype not in _DT or (x.dtype == torch.float32 and out_dtype != torch.float32):
        raise TypeError(f"output dtype {out_dtype} is not supported for {x.dtype} inputs")
    return _DT[out_dtype]


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _call(dev: torch.device, fn, where: str, *args) -> None:
    """One library call on the current stream of `dev`, with `dev` current."""
    if torch.cuda.current_device() == dev.index:
        code = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if code:
        _abi.check(code, where)


def _workspace(nbytes: int, dev: torch.device) -> torch.Tensor:
    """The zero-filled workspace of this device and stream. A call that is being captured gets one of its own,
    from the graph's memory: graphs captured on one stream may be replayed on several at once."""
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    key = (dev.index, torch.cuda.current_stream(dev).cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


def _scratch(workspace, B: int, T: int, C: int, dev: torch.device):
    """(pointer, bytes, tensor kept alive) of the workspace of a call."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        if workspace.device != dev:
            raise ValueError(f"workspace must be on {dev}, the device of the other arguments")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if T <= _abi.WKV_GATED_TILE:  # one tile: the library uses none
        return 0, 0, None
    need = gated_workspace_size(B, T, C)
    if torch.cuda.current_device() == dev.index:
        ws = _workspace(need, dev)
    else:
        with torch.cuda.device(dev):
            ws = _workspace(need, dev)
    return ws.data_ptr(), ws.numel(), ws


def gated_workspace_size(B: int, T: int, C: int) -> int:
    """Bytes of workspace ``gated_forward`` and ``gated_backward`` need for this shape (host-only)."""
    n = _abi.lib().wkv_gated_workspace_size(int(B), int(T), int(C))
    if n == 0:
        raise ValueError("invalid sizes")
    return int(n)


def gated_checkpoints(x: torch.Tensor) -> torch.Tensor:
    """A tensor for the ``checkpoints`` of ``gated_forward`` over x [B, T, C]: the
    state in front of every 128 tokens, float32 [B, ceil(T / 128), C]."""
    B, T, C = x.shape
    tile = _abi.WKV_GATED_TILE
    return torch.empty((B, (T + tile - 1) // tile, C), dtype=torch.float32, device=x.device)


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
    once, for this operator alone; by default one is kept per stream (and
    allocated anew in a call that is captured into a graph).
    """
    xc, zc, gc = _inputs(x, z, 3, "[B, T, C]", gate)
    B, T, C = x.shape
    dev = x.device
    oc = _out_code(x, out_dtype or (x.dtype if out is None else out.dtype))
    if out is None:
        out = torch.empty((B, T, C), dtype=out_dtype or x.dtype, device=dev)
    else:
        _tensor(out, "out", dev, (B, T, C), out_dtype or out.dtype)
    if state is not None:
        _tensor(state, "state", dev, (B, C), torch.float32)
    if state_out is None:
        state_out = torch.empty((B, C), dtype=torch.float32, device=dev)
    else:
        _tensor(state_out, "state_out", dev, (B, C), torch.float32)
    if checkpoints is not None:
        tile = _abi.WKV_GATED_TILE
        _tensor(checkpoints, "checkpoints", dev, (B, (T + tile - 1) // tile, C), torch.float32)
    ws, nws, keep = _scratch(workspace, B, T, C, dev)
    xs, zs = x.stride(), z.stride()
    _call(dev, _abi.lib().wkv_gated_forward, "wkv_gated_forward", B, T, C, x.data_ptr(), xc, xs[0], xs[1],
          z.data_ptr(), zc, zs[0], zs[1], gc, out.data_ptr(), oc, _ptr(state), state_out.data_ptr(), _ptr(checkpoints),
          ws, nws)
    return out, state_out


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
    xc, zc, gc = _inputs(x, z, 3, "[B, T, C]", gate)
    B, T, C = x.shape
    dev = x.device
    oc = _out_code(x, gout.dtype if isinstance(gout, torch.Tensor) else None)
    _tensor(gout, "gout", dev, (B, T, C), gout.dtype)
    if state is not None:
        _tensor(state, "state", dev, (B, C), torch.float32)
    if dstate is not None:
        _tensor(dstate, "dstate", dev, (B, C), torch.float32)
    tile = _abi.WKV_GATED_TILE
    if checkpoints is not None:
        _tensor(checkpoints, "checkpoints", dev, (B, (T + tile - 1) // tile, C), torch.float32)
    ws, nws, keep = _scratch(workspace, B, T, C, dev)
    xs, zs = x.stride(), z.stride()
    inputs = (B, T, C, x.data_ptr(), xc, xs[0], xs[1], z.data_ptr(), zc, zs[0], zs[1], gc)
    if checkpoints is None and T > tile:
        checkpoints = gated_checkpoints(x)
        _call(dev, _abi.lib().wkv_gated_forward, "wkv_gated_forward", *inputs, 0, oc, _ptr(state), 0,
              checkpoints.data_ptr(), ws, nws)
    dx = torch.empty((B, T, C), dtype=x.dtype, device=dev)
    dz = torch.empty((B, T, C), dtype=z.dtype, device=dev)
    dstate_in = torch.empty((B, C), dtype=torch.float32, device=dev)
    _call(dev, _abi.lib().wkv_gated_backward, "wkv_gated_backward", *inputs, gout.data_ptr(), oc, _ptr(state),
          _ptr(dstate), _ptr(checkpoints), dx.data_ptr(), dz.data_ptr(), dstate_in.data_ptr(), ws, nws)
    return dx, dz, dstate_in


def gated_step(state: torch.Tensor, x: torch.Tensor, z: torch.Tensor, *, gate: str = "sigmoid",
               out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               state_out: Optional[torch.Tensor] = None, inplace: bool = False):
    """One token for S streams: x, z [S, C] (channel axis contiguous), state
    float32 [S, C]. Returns (out [S, C], new state); with ``inplace=True`` the
    state tensor is updated in place and returned."""
    xc, zc, gc = _inputs(x, z, 2, "[S, C]", gate)
    S, C = x.shape
    dev = x.device
    oc = _out_code(x, out_dtype or (x.dtype if out is None else out.dtype))
    _tensor(state, "state", dev, (S, C), torch.float32)
    if out is None:
        out = torch.empty((S, C), dtype=out_dtype or x.dtype, device=dev)
    else:
        _tensor(out, "out", dev, (S, C), out_dtype or out.dtype)
    if inplace:
        state_out = state
    elif state_out is None:
        state_out = torch.empty((S, C), dtype=torch.float32, device=dev)
    else:
        _tensor(state_out, "state_out", dev, (S, C), torch.float32)
    _call(dev, _abi.lib().wkv_gated_step, "wkv_gated_step", S, C, x.data_ptr(), xc, x.stride(0), z.data_ptr(), zc,
          z.stride(0), gc, out.data_ptr(), oc, state.data_ptr(), state_out.data_ptr())
    return out, state_out


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
