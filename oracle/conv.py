"""CPU fp64 oracle of the short causal convolution per channel, its gradients and its form on a pool of windows.

TEST INFRASTRUCTURE: imported by the test suite only; shares no code with the HIP library. One sequence at a time: its
window [W-1, D] before its inputs x [len, D], taps weight [D, W]:
    z_t = b + sum_j w[:, j] u_{t+j} over u = window followed by x,   y = z or z sigmoid(z).
"""
from __future__ import annotations

import numpy as np

from .recurrence import _f64


def sigmoid(z):
    return 0.5 * (1.0 + np.tanh(0.5 * z))


def spans(shape, cu):
    """(row, begin, end) of every sequence of x [B, T, D]."""
    if cu is None:
        return [(b, 0, shape[1]) for b in range(shape[0])]
    cu = np.asarray(cu)
    return [(0, int(cu[n]), int(cu[n + 1])) for n in range(len(cu) - 1)]


def taps(u, w, b):
    W = w.shape[1]
    z = np.zeros((u.shape[0] - (W - 1), u.shape[1])) + (0.0 if b is None else _f64(b))
    for t in range(z.shape[0]):
        for j in range(W):
            z[t] += w[:, j] * u[t + j]
    return z


def forward(x, w, b, window0, cu, silu):
    """y (NaN in the rows that no sequence covers) and the windows behind the sequences."""
    x, w = _f64(x), _f64(w)
    W, D = w.shape[1], x.shape[2]
    y, last = np.full(x.shape, np.nan), []
    for n, (r, i, j) in enumerate(spans(x.shape, cu)):
        u = np.concatenate([np.zeros((W - 1, D)) if window0 is None else _f64(window0)[n], x[r, i:j]])
        z = taps(u, w, b)
        y[r, i:j] = z * sigmoid(z) if silu else z
        last.append(u[len(u) - (W - 1):])
    return y, np.stack(last)


def backward(x, w, b, window0, dy, dlast, cu, silu):
    """dx (NaN in the rows that no sequence covers), dw, db, dwindow0."""
    x, w, dy = _f64(x), _f64(w), _f64(dy)
    W, D = w.shape[1], x.shape[2]
    dx, dw, db, dwin = np.full(x.shape, np.nan), np.zeros_like(w), np.zeros(D), []
    for n, (r, i, j) in enumerate(spans(x.shape, cu)):
        u = np.concatenate([np.zeros((W - 1, D)) if window0 is None else _f64(window0)[n], x[r, i:j]])
        z = taps(u, w, b)
        s = sigmoid(z)
        dz = dy[r, i:j] * (s + z * s * (1 - s) if silu else 1.0)
        du = np.zeros_like(u)
        if dlast is not None:
            du[len(u) - (W - 1):] += _f64(dlast)[n]
        for t in range(j - i):
            for k in range(W):
                du[t + k] += w[:, k] * dz[t]
                dw[:, k] += dz[t] * u[t + k]
        db += dz.sum(0)
        dx[r, i:j] = du[W - 1:]
        dwin.append(du[: W - 1])
    return dx, dw, db, np.stack(dwin)


def run(x, w, b, windows, slots, cu, out_slots, silu):
    """x [T, D] on a pool: y (NaN in the rows that no sequence covers) and the pool afterwards."""
    x, w, windows = _f64(x), _f64(w), _f64(windows)
    T, W = x.shape[0], w.shape[1]
    cu = np.arange(T + 1) if cu is None else np.asarray(cu)
    y, pool = np.full(x.shape, np.nan), windows.copy()
    for n, slot in enumerate(np.asarray(slots)):
        i, j = cu[n], cu[n + 1]
        if not 0 <= slot < windows.shape[0]:
            y[i:j] = 0.0
            continue
        u = np.concatenate([windows[slot], x[i:j]])
        z = taps(u, w, b)
        y[i:j] = z * sigmoid(z) if silu else z
        if out_slots is None and j > i:
            pool[slot] = u[len(u) - (W - 1):]
        for t in range(i, j) if out_slots is not None else ():
            if 0 <= out_slots[t] < windows.shape[0]:
                pool[out_slots[t]] = u[t - i + 1: t - i + W]
    return y, pool
