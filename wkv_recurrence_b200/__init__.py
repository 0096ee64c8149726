"""B200 (sm_100a) implementation of the RWKV time-mixing WKV operator.

The operator is the per-channel decayed weighted mean of "Linear attention
without writing a CUDA kernel", section "The recurrence", carried as a
(numerator, denominator, max_exponent) state. The work runs in libwkv.so
(hand-written CUDA, C ABI in include/wkv.h); this package is its Python
binding:

    out, state = wkv_recurrence_b200.forward(k, v, w, u, state=None)
    out, state = wkv_recurrence_b200.forward_host(k_host, v_host, w, u)  # k, v in host memory
    out, state = wkv_recurrence_b200.step(state, k, v, w, u)
    out, state = wkv_recurrence_b200.gated_forward(x, z, state)          # the gated linear recurrence
    out, state = wkv_recurrence_b200.gated_step(state, x, z)
    y, residual = wkv_recurrence_b200.rms_norm(x, weight, residual)      # of the residual stream
    q, scale, residual = wkv_recurrence_b200.rms_norm_quant(x, weight, residual)

Importing the package does not load the library; the first call does, and
fails loudly if it is missing or no CUDA device is present.
"""

from .api import (WKV, PreparedForward, PreparedStep, WkvError, backward, empty_state, forward,  # noqa: F401
                  forward_host, forward_host_buffer_size, forward_kernel, forward_launches, make_workspace,
                  query_status, step, v6_forward, workspace_size)
from .gated import (Gated, gated_backward, gated_checkpoints, gated_forward, gated_step,  # noqa: F401
                    gated_status, gated_workspace_size)
from .norm import RMSNorm, rms_norm, rms_norm_backward, rms_norm_quant  # noqa: F401

__all__ = ["forward", "forward_host", "forward_host_buffer_size", "step", "backward", "WKV", "v6_forward",
           "workspace_size", "forward_kernel", "forward_launches", "make_workspace", "query_status", "empty_state",
           "PreparedForward", "PreparedStep", "WkvError", "gated_forward", "gated_backward", "gated_step",
           "gated_checkpoints", "gated_workspace_size", "gated_status", "Gated", "rms_norm", "rms_norm_quant",
           "rms_norm_backward", "RMSNorm"]
