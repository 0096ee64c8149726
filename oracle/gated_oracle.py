"""Float64 oracle of the gated linear recurrence and its gradients, with a
running error analysis of an fp32 evaluation.

    h_t = f_t h_{t-1} + i_t x_t     sigmoid: f = sigmoid(z), i = 1 - f;  decay: f = e^{-z}, i = 1

``forward`` and ``backward`` are the definition, token after token.
``allowed_*`` bound how far a correct fp32 evaluation may be from it. With
U = 2^-23 (twice the unit roundoff), per token:
  * rounding: at most four rounded operations on values no larger than A_t, the
    recurrence of the magnitudes: 4 U A_t;
  * the gate: z times log2(e) is rounded twice (constant and product), which
    the exponential turns into a relative error of 2 |z| 2^-24 = |z| U; the
    exponential (2 units), the reciprocal (1), the sum and the product before
    them add less than 8 U. The smaller of f and 1 - f carries that relative
    error; so the token's input i|x| and the state's change min(f, 1 - f) A do;
  * both errors are then carried on by f like the state itself;
  * in gradients 1 - f is held as no less than 2^-126 (a gate of f = 1 is kept
    as that), so dx may be off by 2^-126 |D| and dz by 2^-126 |D| |h - x|.
A scan regroups the same sums (its span products carry the same relative
errors as the factors, and it adds fewer roundings than there are tokens):
the bound is doubled for it.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -23
HELD = 2.0 ** -126


def gates(z, gate):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        if gate == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
        return np.exp(-z), np.ones_like(z)


def _small(z, f, gate):
    """min(f, |1 - f|) (times the gate's relative error gives f's absolute one) and that relative error."""
    zz = np.where(np.isfinite(z), np.abs(z), 0.0)
    m = 1.0 / (1.0 + np.exp(np.clip(z, -700, 700))) if gate == "sigmoid" else np.abs(-np.expm1(-np.asarray(z, np.float64)))
    return np.minimum(f, m) if gate == "sigmoid" else np.where(z >= 0, np.minimum(f, m), f), (zz + 8) * U


def forward(x, z, h0, gate):
    """(out [B, T, C], state [B, C]) in float64."""
    x = np.asarray(x, np.float64)
    f, i = gates(z, gate)
    h = np.zeros(x.shape[::2]) if h0 is None else np.asarray(h0, np.float64)
    out = np.empty_like(x)
    for t in range(x.shape[1]):
        h = f[:, t] * h + i[:, t] * x[:, t]
        out[:, t] = h
    return out, h


def allowed_forward(x, z, h0, gate):
    """Bound on an fp32 evaluation's error of every out_t (and, at the end, of the state)."""
    x = np.abs(np.asarray(x, np.float64))
    f, i = gates(z, gate)
    low, rel = _small(z, f, gate)
    A = np.zeros(x.shape[::2]) if h0 is None else np.abs(np.asarray(h0, np.float64))
    E = np.zeros_like(A)
    out = np.empty_like(x)
    mag = np.empty_like(x)
    for t in range(x.shape[1]):
        add = i[:, t] * x[:, t]
        new = f[:, t] * A + add
        E = f[:, t] * E + 4 * U * new + rel[:, t] * low[:, t] * ((x[:, t] if gate == "sigmoid" else 0) + A)
        A = new
        out[:, t], mag[:, t] = 2 * E, A
    return out, mag


def backward(x, z, h0, g, dstate, gate):
    """(dx, dz, dstate_in) in float64."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    f, i = gates(z, gate)
    out, _ = forward(x, z, h0, gate)
    before = np.empty_like(out)
    before[:, 0] = 0 if h0 is None else h0
    before[:, 1:] = out[:, :-1]
    q = np.zeros(x.shape[::2]) if dstate is None else np.asarray(dstate, np.float64)
    dx, dz = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[1] - 1, -1, -1):
        D = g[:, t] + q
        dx[:, t] = i[:, t] * D
        dz[:, t] = D * (before[:, t] - x[:, t]) * f[:, t] * i[:, t] if gate == "sigmoid" else -D * before[:, t] * f[:, t]
        q = f[:, t] * D
    return dx, dz, q


def allowed_backward(x, z, h0, g, dstate, gate):
    """Bounds on an fp32 evaluation's errors of dx, dz and dstate_in."""
    f, i = gates(z, gate)
    low, rel = _small(z, f, gate)
    Eh, Ah = allowed_forward(x, z, h0, gate)
    ax, ag = np.abs(np.asarray(x, np.float64)), np.abs(np.asarray(g, np.float64))
    eb, ab = np.zeros_like(Eh), np.zeros_like(Ah)
    eb[:, 1:], ab[:, 1:] = Eh[:, :-1], Ah[:, :-1]
    ab[:, 0] = 0 if h0 is None else np.abs(h0)
    q = np.zeros(ax.shape[::2]) if dstate is None else np.abs(np.asarray(dstate, np.float64))
    E = np.zeros_like(q)
    dx, dz = np.empty_like(ax), np.empty_like(ax)
    for t in range(ax.shape[1] - 1, -1, -1):
        D = ag[:, t] + q
        ED = E + U * D
        dx[:, t] = 2 * i[:, t] * ED + (rel[:, t] * low[:, t] + 2 * U * i[:, t] + HELD) * D
        w = f[:, t] * i[:, t]
        span = ab[:, t] + (ax[:, t] if gate == "sigmoid" else 0)
        dz[:, t] = 2 * ED * span * w + D * eb[:, t] * w + D * span * (w * (2 * rel[:, t] + 6 * U) + HELD)
        E = f[:, t] * ED + 3 * U * f[:, t] * D + rel[:, t] * low[:, t] * D
        q = f[:, t] * D
    return dx, dz, 2 * E
