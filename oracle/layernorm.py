"""CPU fp64 oracle of layer norm and its gradients.

TEST INFRASTRUCTURE: imported by the test suite only; shares no code with the HIP library. Per row s [d], m and v its mean
and variance: xh = (s - m) / sqrt(v + eps), y = w xh + b. The backward pass is the transposed Jacobian, written out as
dx_i = sum_j g_j dxh_j/ds_i with dxh_j/ds_i = (delta_ij - 1/d - xh_i xh_j / d) / sqrt(v + eps), g = w dy.
"""
from __future__ import annotations

import numpy as np

from .recurrence import _f64


def normalise(s, eps):
    s = _f64(s)
    c = s - s.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return c * rstd, rstd


def forward(s, w, b, eps):
    y, _ = normalise(s, eps)
    if w is not None:
        y = y * _f64(w)
    return y if b is None else y + _f64(b)


def backward(s, dy, w, ds, eps):
    """dx, dw, db for s, dy [rows, d]."""
    xh, rstd = normalise(s, eps)
    dy = _f64(dy)
    d = xh.shape[-1]
    g = dy if w is None else dy * _f64(w)
    dx = rstd * (g - g.sum(-1, keepdims=True) / d - xh * (xh * g).sum(-1, keepdims=True) / d)   # the Jacobian times g, row by row
    if ds is not None:
        dx = dx + _f64(ds)
    return dx, (dy * xh).sum(0), dy.sum(0)
