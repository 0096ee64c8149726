"""Float64 oracle of the RMS norm by groups, its e4m3 scales and its gradients,
with bounds on the error of an fp32 evaluation (U = 2^-24, fp32's half step).

Sums of n fp32 products, however they are grouped, are off by at most n U of
the sum of the magnitudes; in the trees and lanes used here a sum of D terms
passes at most 8 K + 20 additions (K vectors of 8 columns per thread, then
shuffles), D / 32 + 20 in the kernels that walk a row. ``_depth`` takes the
larger of the two.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def _depth(D):
    return min(D, 32 + D / 32) + 20


def rms(s, weight, eps, groups):
    """y and r = (mean s^2 + eps)^-1/2 [N, groups]."""
    s = np.asarray(s, np.float64)
    N, C = s.shape
    h = s.reshape(N, groups, -1)
    r = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return (h * r[..., None]).reshape(N, C) * np.asarray(weight, np.float64), r


def rel_y(D):
    """Relative error of y: half that of the mean of squares, the square root, quotient and two products."""
    return (_depth(D) / 2 + 6) * U


def scales(y, block):
    N, C = y.shape
    b = block or C
    top = np.abs(y.reshape(N, C // b, b)).max(-1)
    return np.where(top > 0, top / 448.0, 1.0)


def backward(gy, s, weight, gs, eps, groups):
    """(ds, dweight, bound on ds, bound on dweight)."""
    gy, s, w = (np.asarray(t, np.float64) for t in (gy, s, weight))
    N, C = s.shape
    D = C // groups
    _, r = rms(s, w, eps, groups)
    h, p = s.reshape(N, groups, D), (gy * w).reshape(N, groups, D)
    m = (p * h).mean(-1) * r * r
    d = r[..., None] * (p - h * m[..., None])
    # |p| and |s m| with m's sums taken over magnitudes
    mm = (np.abs(p * h)).mean(-1) * r * r
    mag = r[..., None] * (np.abs(p) + np.abs(h) * mm[..., None])
    bound = mag.reshape(N, C) * (3 * _depth(D) + 16) * U
    ds = d.reshape(N, C)
    if gs is not None:
        ds = ds + np.asarray(gs, np.float64)
        bound = bound + np.abs(ds) * U
    unit = (h * r[..., None]).reshape(N, C)
    dw = (gy * unit).sum(0)
    # a part adds its rows one after the other, at most N of them, then the parts are added
    dw_bound = np.abs(gy * unit).sum(0) * (min(N, 600) + 200 + _depth(D)) * U
    return ds, dw, bound, dw_bound
