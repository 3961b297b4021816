"""CPU fp64 oracle of the backward pass of the channel-wise rule: the adjoint of the token step of kda.py.

TEST INFRASTRUCTURE: imported by the test suite only; shares no code with the HIP library.

Forward step of one head: Sa = S Diag(a), a = exp(g); u = v - Sa k; S' = Sa + beta u k^T; o = S' q. Backward, from dS'
(the gradient reaching S' from later tokens and the final state) and do:
    dS' += do q^T;  dq = S'^T do;  de = dS' k (the gradient of beta u);  dv = beta de;  dbeta = de . u
    dk = dS'^T (beta u) - Sa^T dv;  dSa = dS' - dv k^T;  dg = a * colsum(dSa * S) = colsum(dSa * Sa);  dS = dSa Diag(a)
"""
from __future__ import annotations

import numpy as np

from .recurrence import _f64, segments


def backward(q, k, v, g, beta, do, h0=None, dhT=None, cu_seqlens=None):
    """Arguments as kda.forward's, do like o, dhT like hT. Returns dq, dk, dv, dg, dbeta, dh0."""
    q, k, v, g, beta, do, h0, dhT = (_f64(x) for x in (q, k, v, g, beta, do, h0, dhT))
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    segs = segments(B, T, cu_seqlens)
    q, k, v, g, beta, do = (x.reshape((1, B * T) + x.shape[2:]) for x in (q, k, v, g, beta, do))
    dq, dk_, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(g)
    dv_, db = np.zeros_like(v), np.zeros_like(beta)
    dh0 = np.zeros((len(segs), H, dv, dk))
    b = 0
    for n, (t0, t1) in enumerate(segs):
        S = np.zeros((H, dv, dk)) if h0 is None else h0[n].copy()
        kept = []
        for t in range(t0, t1):
            Sa = S * np.exp(g[b, t])[:, None, :]
            u = v[b, t] - np.einsum("hvk,hk->hv", Sa, k[b, t])
            S = Sa + beta[b, t][:, None, None] * u[:, :, None] * k[b, t][:, None, :]
            kept.append((Sa, u, S))
        dS = np.zeros((H, dv, dk)) if dhT is None else dhT[n].copy()
        for t in reversed(range(t0, t1)):
            Sa, u, S = kept[t - t0]
            dS = dS + do[b, t][:, :, None] * q[b, t][:, None, :]
            dq[b, t] = np.einsum("hvk,hv->hk", S, do[b, t])
            de = np.einsum("hvk,hk->hv", dS, k[b, t])
            dv_[b, t] = beta[b, t][:, None] * de
            db[b, t] = (de * u).sum(-1)
            dk_[b, t] = (np.einsum("hvk,hv->hk", dS, beta[b, t][:, None] * u)
                         - np.einsum("hvk,hv->hk", Sa, dv_[b, t]))
            dSa = dS - dv_[b, t][:, :, None] * k[b, t][:, None, :]
            dg[b, t] = (dSa * Sa).sum(1)
            dS = dSa * np.exp(g[b, t])[:, None, :]
        dh0[n] = dS
    return (*(x.reshape((B, T) + x.shape[2:]) for x in (dq, dk_, dv_, dg, db)), dh0)
