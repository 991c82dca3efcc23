"""fp64 CPU oracle of the gated delta rule (test infrastructure only: the
tests and the smoke check may import it; the HIP library never does).

Per sequence and head, with S in R^{P x N} starting at the initial state:

    Sd_t = exp(g_t) S_{t-1},  e_t = v_t - Sd_t k_t,  S_t = Sd_t + beta_t e_t k_t^T,  o_t = scale S_t q_t

token by token.  The adjoint is the same loop read backwards: with D the
gradient of S_t (from later tokens, plus scale dout_t q_t^T),

    dq_t = scale S_t^T dout_t,  du = D k_t,  dbeta_t = du . e_t,  dv_t = beta_t du,
    dk_t = D^T (beta_t e_t) - Sd_t^T dv_t,
    D' = D - dv_t k_t^T,  dg_t = <D', Sd_t>,  D <- exp(g_t) D'.

Arrays are laid out as include/gated_delta.h says; everything is numpy
float64, vectorised over the heads.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np


def sequences(b: int, L: int, seq_idx: Optional[np.ndarray]) -> list[tuple[int, int, int]]:
    """(batch row, first row, end) of every sequence, in order."""
    out = []
    for i in range(b):
        cuts = [0] + ([] if seq_idx is None else [t for t in range(1, L) if seq_idx[i, t] != seq_idx[i, t - 1]]) + [L]
        out += [(i, cuts[j], cuts[j + 1]) for j in range(len(cuts) - 1)]
    return out


def _heads(x, rep):
    return np.repeat(np.asarray(x, np.float64), rep, axis=2)


def forward(q, k, v, g, beta, initial_states=None, seq_idx=None, scale=None):
    """dict of o and final_states (fp64)."""
    v, g, beta = (np.asarray(x, np.float64) for x in (v, g, beta))
    b, L, H, P = v.shape
    N = q.shape[3]
    scale = 1.0 / math.sqrt(N) if scale is None else scale
    q, k = _heads(q, H // q.shape[2]), _heads(k, H // k.shape[2])
    seqs = sequences(b, L, seq_idx)
    o, final = np.zeros_like(v), np.zeros((len(seqs), H, P, N))
    for s, (i, t0, t1) in enumerate(seqs):
        S = np.zeros((H, P, N)) if initial_states is None else np.asarray(initial_states[s], np.float64).copy()
        for t in range(t0, t1):
            S = S * np.exp(g[i, t])[:, None, None]
            e = v[i, t] - np.einsum("hpn,hn->hp", S, k[i, t])
            S = S + (beta[i, t][:, None] * e)[:, :, None] * k[i, t][:, None, :]
            o[i, t] = scale * np.einsum("hpn,hn->hp", S, q[i, t])
        final[s] = S
    return {"o": o, "final_states": final}


def backward(q, k, v, g, beta, dout, initial_states=None, seq_idx=None, d_final_states=None, scale=None):
    """dict of dq, dk, dv, dg, dbeta, d_initial_states (fp64) of l = sum dout o + sum d_final_states final_states."""
    v, g, beta, dout = (np.asarray(x, np.float64) for x in (v, g, beta, dout))
    b, L, H, P = v.shape
    G, N = q.shape[2], q.shape[3]
    scale = 1.0 / math.sqrt(N) if scale is None else scale
    q, k = _heads(q, H // G), _heads(k, H // G)
    seqs = sequences(b, L, seq_idx)
    dq, dk, dv, dg, db = (np.zeros_like(x) for x in (q, k, v, g, beta))
    dinit = np.zeros((len(seqs), H, P, N))
    for s, (i, t0, t1) in enumerate(seqs):
        S = np.zeros((H, P, N)) if initial_states is None else np.asarray(initial_states[s], np.float64).copy()
        saved = []
        for t in range(t0, t1):
            Sd = S * np.exp(g[i, t])[:, None, None]
            e = v[i, t] - np.einsum("hpn,hn->hp", Sd, k[i, t])
            S = Sd + (beta[i, t][:, None] * e)[:, :, None] * k[i, t][:, None, :]
            saved.append((Sd, e, S))
        D = np.zeros((H, P, N)) if d_final_states is None else np.asarray(d_final_states[s], np.float64).copy()
        for t in range(t1 - 1, t0 - 1, -1):
            Sd, e, S = saved.pop()
            D = D + scale * dout[i, t][:, :, None] * q[i, t][:, None, :]
            dq[i, t] = scale * np.einsum("hpn,hp->hn", S, dout[i, t])
            du = np.einsum("hpn,hn->hp", D, k[i, t])
            db[i, t] = (du * e).sum(-1)
            dv[i, t] = beta[i, t][:, None] * du
            dk[i, t] = np.einsum("hpn,hp->hn", D, beta[i, t][:, None] * e) - np.einsum("hpn,hp->hn", Sd, dv[i, t])
            D = D - dv[i, t][:, :, None] * k[i, t][:, None, :]
            dg[i, t] = (D * Sd).sum((-1, -2))
            D = D * np.exp(g[i, t])[:, None, None]
        dinit[s] = D
    fold = lambda x: x.reshape(b, L, G, H // G, N).sum(3)  # noqa: E731
    return {"dq": fold(dq), "dk": fold(dk), "dv": dv, "dg": dg, "dbeta": db, "d_initial_states": dinit}


def step(q, k, v, g, beta, states, state_indices=None, scale=None):
    """(o, states) of delta_step: the rows in order, rows without a state of the pool empty."""
    states = np.asarray(states, np.float64).copy()
    o = np.zeros(np.shape(v))
    for i in range(len(v)):
        at = i if state_indices is None else int(state_indices[i])
        if not 0 <= at < len(states):
            continue
        row = lambda x: np.asarray(x)[i:i + 1]  # noqa: E731
        r = forward(row(q), row(k), row(v), row(g), row(beta), states[at][None], None, scale)
        o[i], states[at] = r["o"][0], r["final_states"][0]
    return o, states
