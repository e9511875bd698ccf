"""Whole sequences on dense states, their gradients, and trees of drafted tokens, in
float64 (oracle).

One token of any form, with a its decay (a scalar per head, KDA: one per channel):

    S' = Diag(a) S,  w = beta (v - S'^T k)  (Mamba-2: w = beta v),  S+ = S' + k w^T,  o = S+^T q

which is ``recurrences.dense_step`` with the written value w named.  The gradients are
the adjoint of exactly these four lines, token by token from the last to the first.

Arrays of one sequence: q, k (T, H, d_k), v (T, H, d_v), alpha (T, H) or (T, H, d_k),
beta (T, H), states (H, d_k, d_v).  Shared key heads are repeated by the caller.
"""

from __future__ import annotations

import numpy as np

from workloads import FORM_KDA, FORM_MAMBA2


def _decay(form, alpha_t):
    a = np.asarray(alpha_t, dtype=np.float64)
    return a[..., :, None] if form == FORM_KDA else a[..., None, None]


def step(form, S, k, v, alpha, beta):
    """One token for states (..., d_k, d_v): returns (S', v - S'^T k or v, w, S+)."""
    Sd = _decay(form, alpha) * S
    r = v if form == FORM_MAMBA2 else v - np.einsum("...i,...ij->...j", k, Sd)
    w = np.asarray(beta)[..., None] * r
    return Sd, r, w, Sd + k[..., :, None] * w[..., None, :]


def scan(form, q, k, v, alpha, beta, S0):
    """o (T, H, d_v) and the final states; S0 (H, d_k, d_v)."""
    S = np.array(S0, dtype=np.float64)
    o = np.zeros(v.shape)
    for t in range(v.shape[0]):
        S = step(form, S, k[t], v[t], alpha[t], beta[t])[3]
        o[t] = np.einsum("hij,hi->hj", S, q[t])
    return o, S


def scan_backward(form, q, k, v, alpha, beta, S0, do, dS_out):
    """Gradients dq, dk, dv, dlog_alpha (= alpha dL/dalpha), dbeta, dS0 of ``scan``."""
    T = v.shape[0]
    kept, S = [], np.array(S0, dtype=np.float64)
    for t in range(T):
        kept.append(step(form, S, k[t], v[t], alpha[t], beta[t]))
        S = kept[-1][3]
    G = np.array(dS_out, dtype=np.float64)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dla, dbeta = np.zeros(np.shape(alpha)), np.zeros(np.shape(beta))
    for t in reversed(range(T)):
        Sd, r, w, Sn = kept[t]
        dq[t] = np.einsum("hij,hj->hi", Sn, do[t])
        G = G + q[t][:, :, None] * do[t][:, None, :]
        dw = np.einsum("hij,hi->hj", G, k[t])
        dk[t] = np.einsum("hij,hj->hi", G, w)
        dv[t] = np.asarray(beta[t])[:, None] * dw
        dbeta[t] = np.sum(r * dw, axis=-1)
        if form != FORM_MAMBA2:
            dk[t] -= np.einsum("hij,hj->hi", Sd, dv[t])
            G = G - k[t][:, :, None] * dv[t][:, None, :]
        dl = np.sum(G * Sd, axis=-1)
        dla[t] = dl if form == FORM_KDA else dl.sum(axis=-1)
        G = _decay(form, alpha[t]) * G
    return dq, dk, dv, dla, dbeta, G


def tree(form, root, parent, q, k, v, alpha, beta):
    """One request's tree: root (H, d_k, d_v), parent (N,), token arrays (N, H, ..).
    Returns o, w (zeros at unused nodes) and the node states (None at unused ones)."""
    o, w, states = np.zeros(v.shape), np.zeros(v.shape), []
    for t, p in enumerate(parent):
        S = None if p < -1 or p >= t else (root if p == -1 else states[p])
        if S is None:
            states.append(None)
            continue
        _, _, w[t], Sn = step(form, S, k[t], v[t], alpha[t], beta[t])
        o[t] = np.einsum("hij,hi->hj", Sn, q[t])
        states.append(Sn)
    return o, w, states


def path(parent, leaf):
    """The nodes from the root to ``leaf`` in order ([] for a negative leaf)."""
    out = []
    while leaf >= 0:
        out.append(leaf)
        leaf = parent[leaf]
    return out[::-1]
