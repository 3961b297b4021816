"""CPU fp64 oracle of the per-head norm of queries and keys with the rotary rotation.

TEST INFRASTRUCTURE: imported by the test suite only; shares no code with the HIP library.

For a row x [d] of a token at position p, n = 1 ("l2") or d ("rms"):
    m = sum x^2 / n + eps,   y = scale * R(p) (w * x / sqrt(m)),
R(p): channels a, b of pair j turned by p * inv_freq[j] and scaled by rope_scale; pair j is (j, j + rot/2) in the
half layout, (2j, 2j + 1) in the interleaved one. The backward pass is the transposed Jacobian, written out:
    g = scale * R^T dy,   dw = sum xh g,   dx = w g / sqrt(m) - x (w g . x) / (n m^{3/2}).
"""
from __future__ import annotations

import numpy as np


def rotation(positions, inv_freq, layout, rope_scale, d):
    """The matrices R [tokens, d, d]."""
    pos = np.asarray(positions, dtype=np.float64).reshape(-1)
    R = np.zeros((pos.size, d, d))
    R[:, np.arange(d), np.arange(d)] = 1.0
    if inv_freq is None:
        return R
    f = np.asarray(inv_freq, dtype=np.float64)
    half = f.size
    for j in range(half):
        a, b = (j, j + half) if layout == "half" else (2 * j, 2 * j + 1)
        c, s = rope_scale * np.cos(pos * f[j]), rope_scale * np.sin(pos * f[j])
        R[:, a, a], R[:, a, b], R[:, b, a], R[:, b, b] = c, -s, s, c
    return R


def forward(x, w, R, norm, eps, scale):
    """x [tokens, heads, d] -> y."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[-1] if norm == "rms" else 1
    z = x / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)
    if w is not None:
        z = z * np.asarray(w, dtype=np.float64)
    return scale * np.einsum("tij,thj->thi", R, z)


def backward(x, dy, w, R, norm, eps, scale):
    """Gradients dx [tokens, heads, d] and dw [d]."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    n = x.shape[-1] if norm == "rms" else 1
    m = (x * x).sum(-1, keepdims=True) / n + eps
    g = scale * np.einsum("tji,thj->thi", R, dy)
    dw = (g * x / np.sqrt(m)).sum((0, 1))
    if w is not None:
        g = g * np.asarray(w, dtype=np.float64)
    return g / np.sqrt(m) - x * (g * x).sum(-1, keepdims=True) / (n * m ** 1.5), dw
