"""CPU fp64 oracle of the recurrent form on a pool of states.

TEST INFRASTRUCTURE: imported by the test suite only; shares no code with the HIP library. Each sequence's run of
tokens goes through the token step of kda.py (a scalar gate is the same decay in every channel).
"""
from __future__ import annotations

import numpy as np

from .kda import step_heads
from .recurrence import _f64


def run(q, k, v, g, beta, states, slots, cu_seqlens=None, out_slots=None):
    """q, k [T,H,dk], v [T,HV,dv], g [T,HV] or [T,HV,dk], beta [T,HV], states [n_slots,HV,dv,dk]. Returns o [T,HV,dv]
    with NaN in the rows that no sequence covers, and the pool afterwards."""
    q, k, v, g, beta, states = (_f64(x) for x in (q, k, v, g, beta, states))
    T, H, dk = q.shape
    HV = v.shape[1]
    head = np.arange(HV) // (HV // H)
    if g.ndim == 2:
        g = np.repeat(g[..., None], dk, -1)
    cu = np.arange(T + 1) if cu_seqlens is None else np.asarray(cu_seqlens)
    o = np.full((T, HV, v.shape[2]), np.nan)
    out = states.copy()
    for n, slot in enumerate(np.asarray(slots)):
        t0, t1 = cu[n], cu[n + 1]
        if not 0 <= slot < states.shape[0]:
            o[t0:t1] = 0.0
            continue
        S = states[slot]
        for t in range(t0, t1):
            S, o[t] = step_heads(S, q[t][head], k[t][head], v[t], g[t], beta[t])
            if out_slots is not None and 0 <= out_slots[t] < states.shape[0]:
                out[out_slots[t]] = S
        if out_slots is None and t1 > t0:
            out[slot] = S
    return o, out
