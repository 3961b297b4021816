"""CPU fp64 oracle of the gated linear recurrence per channel, its gradients, its form on a pool of states, and a bound on what
fp32 arithmetic may add.

TEST INFRASTRUCTURE: imported by the test suite only; shares no code with the HIP library. Token by token:
    h_t = a_t h_{t-1} + b_t,   a = exp(g),   b = x or (blend) (1 - a) x;
backward D_t = dh_t + E_{t+1}, E_t = a_t D_t, dx = D or (1 - a) D, dg = E (h_{t-1} [- x]).

The bound: let u = 2^-24. In a step, a is off by (1.5 |g| + 3) u of itself (the product g log2 e, the exponential), 1 - a by 12 u
(the series: nine roundings; past |g| = 1/2, at most (1.5 |g| + 3) a / (1 - a) + 1 < 8), products and sums by a few u of the magnitudes.
With hbar the recurrence of magnitudes (hbar_t = a hbar_{t-1} + |b_t|), a step adds at most (2 |g| + 16) u hbar_t, and what was off before
decays with a. Evaluating stretches as maps first and joining them takes each step's a once more in another order: twice that. A map's factor goes by
the sum G of its n gates, at most 3 additions in a group of four tokens, 8 over groups and 8 over waves one after another, each off by u |G| at most: with
|G| < 88 (beyond, it is taken for zero) that is less than the 32 n u + 4 |G| u which its steps have.
Below 2^-126 fp32 has no full digits and results may be taken for zero: an exponential (g < -87) or a product is then off by 2^-126
itself, whatever its size, so every step adds 4 (1 + hbar) 2^-126, and a product with a factor m that much times m.
"""
from __future__ import annotations

import numpy as np

from .conv import spans
from .recurrence import _f64

U = 2.0 ** -24
TINY = 2.0 ** -126


def _steps(x, g, blend):
    a = np.exp(g)
    return a, (-np.expm1(g) * x if blend else x)


def forward(x, g, h0, cu, blend):
    """h (NaN in the rows that no sequence covers), hT and their error bounds."""
    x, g = _f64(x), _f64(g)
    D = x.shape[2]
    h, err = np.full(x.shape, np.nan), np.zeros(x.shape)
    last, lerr = [], []
    for n, (r, i, j) in enumerate(spans(x.shape, cu)):
        s = np.zeros(D) if h0 is None else _f64(h0)[n]
        bar, e = np.abs(s), np.zeros(D)
        a, b = _steps(x[r, i:j], g[r, i:j], blend)
        with np.errstate(invalid="ignore"):
            for t in range(j - i):
                s = a[t] * s + b[t]
                bar = a[t] * bar + np.abs(b[t])
                e = a[t] * e + (2 * np.where(np.isfinite(g[r, i + t]), np.abs(g[r, i + t]), 0) + 16) * U * bar + 4 * TINY * (1 + bar)
                h[r, i + t], err[r, i + t] = s, 2 * e
        last.append(s)
        lerr.append(2 * e)
    return h, np.stack(last), err, np.stack(lerr)


def backward(x, g, h0, dh, dhT, cu, blend):
    """dx, dg (NaN in the rows that no sequence covers), dh0, then their error bounds."""
    x, g, dh = _f64(x), _f64(g), _f64(dh)
    D = x.shape[2]
    h, _, herr, _ = forward(x, g, h0, cu, blend)
    dx, dg = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    dxe, dge = np.zeros(x.shape), np.zeros(x.shape)
    first, ferr = [], []
    for n, (r, i, j) in enumerate(spans(x.shape, cu)):
        start = np.zeros(D) if h0 is None else _f64(h0)[n]
        E = np.zeros(D) if dhT is None else _f64(dhT)[n]
        bar, e = np.abs(E), np.zeros(D)
        a, _ = _steps(x[r, i:j], g[r, i:j], blend)
        keep = -np.expm1(g[r, i:j])
        for t in reversed(range(j - i)):
            Dt, Dbar = dh[r, i + t] + E, np.abs(dh[r, i + t]) + bar
            before, berr = (h[r, i + t - 1], herr[r, i + t - 1]) if t else (start, np.zeros(D))
            if blend:
                before = before - x[r, i + t]
            dx[r, i + t] = keep[t] * Dt if blend else Dt
            dxe[r, i + t] = (keep[t] if blend else 1.0) * (2 * e + 16 * U * Dbar) + 4 * TINY * (1 + Dbar)
            E, bar = a[t] * Dt, a[t] * Dbar
            e = a[t] * e + (2 * np.where(np.isfinite(g[r, i + t]), np.abs(g[r, i + t]), 0) + 16) * U * bar + 4 * TINY * (1 + Dbar)
            dg[r, i + t] = E * before
            mag = np.abs(before) + (2 * np.abs(x[r, i + t]) if blend else 0)
            dge[r, i + t] = 2 * e * mag + bar * (berr + 4 * U * mag) + 4 * TINY
        first.append(E)
        ferr.append(2 * e)
    return dx, dg, np.stack(first), dxe, dge, np.stack(ferr)


def run(x, g, states, slots, cu, out_slots, blend):
    """x, g [T, D] on a pool: h (NaN in the rows that no sequence covers), the pool afterwards, and their error bounds."""
    x, g, states = _f64(x), _f64(g), _f64(states)
    T = x.shape[0]
    cu = np.arange(T + 1) if cu is None else np.asarray(cu)
    h, err = np.full(x.shape, np.nan), np.zeros(x.shape)
    pool, perr = states.copy(), np.zeros(states.shape)
    for n, slot in enumerate(np.asarray(slots)):
        i, j = int(cu[n]), int(cu[n + 1])
        if not 0 <= slot < states.shape[0]:
            h[i:j] = 0.0
            continue
        if j == i:
            continue
        y, last, e, le = forward(x[None, i:j], g[None, i:j], states[slot][None], None, blend)
        h[i:j], err[i:j] = y[0], e[0]
        if out_slots is None:
            pool[slot], perr[slot] = last[0], le[0]
        else:
            for t in range(i, j):
                if 0 <= out_slots[t] < states.shape[0]:
                    pool[out_slots[t]], perr[out_slots[t]] = y[0, t - i], e[0, t - i]
    return h, pool, err, perr
