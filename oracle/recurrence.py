"""fp64 CPU oracle of the gated linear recurrence of include/linear_recurrence.h
(test infrastructure only), row by row, with a bound of what float32 arithmetic
may add to every element.

The bounds carry an absolute error along with every value.  A decay, an input
factor and their derivatives are off by at most K of their size,

    K = (16 + 8 |l| + 2 |g|) 2^-24

(l the log decay): an exponential of x is off by (2 + 2 |x|) 2^-24, a
reciprocal and a root by 2^-23, each of the at most eight further roundings by
2^-24, and the series of 1 - exp by 2^-22.  A row adds K of each product to what
the rows before it left.

Below 2^-126 float32 has fewer bits or none: a sigmoid or a log decay l there
counts as any value up to it.  sqrt(1 - a^2) is sqrt(2 |l|) there, so with
|decay| <= 8 (l = decay sigmoid) it may be off by M = sqrt(2 * 9) 2^-63 < 2^-60,
and so may |dm l| = m / 2, which is what reaches dg; ddecay gets |dm sigmoid|,
off by M / |decay|.
"""
from __future__ import annotations

import numpy as np

ULP = 2.0 ** -24
LOST = 2.0 ** -60   # M


def _sigmoids(x):
    e = np.exp(-np.abs(x))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(x < 0, small, big), np.where(x < 0, big, small)


def _gates(g, decay, gate, input_scale):
    s, rest = _sigmoids(g)
    if gate == "log":
        la, dg = g, np.ones_like(g)
    elif gate == "sigmoid":
        la, dg = np.log(s), rest
    else:
        la, dg = decay * s, decay * s * rest
    a = s if gate == "sigmoid" else np.exp(la)
    one = rest if gate == "sigmoid" else -np.expm1(la)
    if input_scale == "one":
        m, dm = np.ones_like(a), np.zeros_like(a)
    elif input_scale == "complement":
        m, dm = one, -a
    else:
        m = np.sqrt(one * (1 + a))
        dm = -a * a / np.where(m == 0, np.inf, m)
    # the size of log decays that matters: those of lost states are -inf
    small = np.maximum(la, -104.0)
    K = (16 + 8 * np.abs(small) + (0 if gate == "log" else 2 * np.abs(g))) * ULP
    return a, m, dm, dg, s, K


def starts_of(shape, seq_idx):
    """(rows of the first of each sequence, in row order) over the flattened rows"""
    b, L = shape[:2]
    first = np.zeros((b, L), bool)
    first[:, 0] = True
    if seq_idx is not None:
        first[:, 1:] |= np.asarray(seq_idx)[:, 1:] != np.asarray(seq_idx)[:, :-1]
    return np.flatnonzero(first.reshape(-1))


def forward(x, g, in_gate=None, decay=None, h0=None, seq_idx=None, gate="sigmoid", input_scale="one"):
    """dict of y, final_states and bounds y_err, final_err"""
    return _run(x, g, in_gate, decay, h0, seq_idx, gate, input_scale)[0]


def _run(x, g, in_gate, decay, h0, seq_idx, gate, input_scale):
    shape, C = x.shape, x.shape[-1]
    x, g = x.reshape(-1, C), g.reshape(-1, C)
    a, m, dm, dg, sg, K = _gates(g, decay, gate, input_scale)
    if in_gate is not None:
        in_gate = in_gate.reshape(-1, C)
        si, ri = _sigmoids(in_gate)
        K = K + 2 * np.abs(in_gate) * ULP
    else:
        si, ri = np.ones_like(x), np.zeros_like(x)
    u = x * si
    starts = starts_of(shape, seq_idx)
    edges = np.append(starts, len(x))
    M = LOST if input_scale == "unit" else 0.0
    h, err, prev, prev_err = (np.zeros_like(x) for _ in range(4))
    for s in range(len(starts)):
        state = np.zeros(C) if h0 is None else h0[s].copy()
        e = np.zeros(C)
        for t in range(edges[s], edges[s + 1]):
            prev[t], prev_err[t] = state, e
            e = a[t] * e + K[t] * (np.abs(a[t] * state) + np.abs(m[t] * u[t])) + M * np.abs(u[t])
            state = a[t] * state + m[t] * u[t]
            h[t], err[t] = state, e
    last = edges[1:] - 1
    out = {"y": h.reshape(shape), "y_err": err.reshape(shape), "final_states": h[last], "final_err": err[last]}
    return out, (x, a, m, dm, dg, sg, si, ri, u, K, prev, prev_err, edges)


def backward(x, g, in_gate, decay, dy, h0=None, seq_idx=None, d_final=None, gate="sigmoid", input_scale="one"):
    """dict of dx, dg, d_in_gate, ddecay, d_initial_states, each with a bound under name + "_err" """
    shape, C = x.shape, x.shape[-1]
    _, (x, a, m, dm, dg, sg, si, ri, u, K, prev, prev_err, edges) = _run(x, g, in_gate, decay, h0, seq_idx, gate, input_scale)
    dy = dy.reshape(-1, C)
    M = LOST if input_scale == "unit" else 0.0
    e, ee = np.zeros_like(x), np.zeros_like(x)
    d0, d0e = np.zeros((len(edges) - 1, C)), np.zeros((len(edges) - 1, C))
    for s in range(len(edges) - 1):
        c, ce = np.zeros(C), np.zeros(C)
        for t in range(edges[s + 1] - 1, edges[s] - 1, -1):
            e[t], ee[t] = dy[t] + c, ce
            if d_final is not None and t == edges[s + 1] - 1:
                e[t] = e[t] + d_final[s]
            ee[t] = ee[t] + 2 * ULP * (np.abs(dy[t]) + np.abs(e[t]))
            c, ce = a[t] * e[t], a[t] * ee[t] + K[t] * np.abs(a[t] * e[t])
        d0[s], d0e[s] = c, ce
    add = np.zeros_like(x) if input_scale == "one" else dm * u   # a factor of one has no share, whatever x is
    inner = a * prev + add
    inner_err = a * prev_err + K * (np.abs(a * prev) + 2 * np.abs(add))
    dl, dle = e * inner, ee * np.abs(inner) + np.abs(e) * inner_err
    du, due = e * m, ee * np.abs(m) + K * np.abs(e * m) + M * np.abs(e)
    lost = M * np.abs(e * u)
    out = {"dx": du * si, "dx_err": due * si + K * np.abs(du * si), "dg": dl * dg, "dg_err": dle * np.abs(dg) + 2 * K * np.abs(dl * dg) + lost,
           "d_initial_states": d0, "d_initial_states_err": d0e}
    out["d_in_gate"] = du * u * ri
    out["d_in_gate_err"] = due * np.abs(u * ri) + 3 * K * np.abs(du * u * ri)
    for k in ("dx", "dg", "d_in_gate"):
        out[k], out[k + "_err"] = out[k].reshape(shape), out[k + "_err"].reshape(shape)
    out["ddecay"] = (dl * sg).sum(0)
    # 64 rows are summed in float32 before the chunks' sums meet in double
    out["ddecay_err"] = ((dle + K * np.abs(dl)) * sg).sum(0) + 64 * ULP * np.abs(dl * sg).sum(0)
    if gate == "decay" and M:
        out["ddecay_err"] += lost.sum(0) / np.where(decay == 0, np.inf, np.abs(decay))
    return out
