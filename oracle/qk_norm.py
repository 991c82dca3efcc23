"""fp64 CPU oracle of the per-head norm with rotation of include/qk_norm.h
(test infrastructure only).

    z = w x r,  r = (mean x^2 + eps)^-1/2 or (sum x^2 + eps)^-1/2,  y = R z

with R the turn of z's first 2 len(inv_freq) values, pair by pair.  R is
orthogonal, so dz = R^T dy; then dw = sum dz x r and, with m = N or 1,
dx = r w dz - x r^3 (sum w dz x) / m.
"""
from __future__ import annotations

import numpy as np


def _turn(z, positions, inv_freq, interleaved, sign):
    if inv_freq is None or len(inv_freq) == 0:
        return z
    half = len(inv_freq)
    t = sign * np.asarray(positions, np.float64)[:, :, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(t), np.sin(t)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out = z.copy()
    a, b = z[..., ia], z[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def _parts(x, weight, positions, eps, norm):
    x = np.asarray(x, np.float64)
    m = x.shape[-1] if norm == "rms" else 1
    r = ((x * x).sum(-1, keepdims=True) / m + eps) ** -0.5
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    if positions is None:
        positions = np.broadcast_to(np.arange(x.shape[1]), x.shape[:2])
    return x, m, r, w, positions


def forward(x, weight=None, positions=None, inv_freq=None, eps=1e-6, norm="rms", interleaved=False):
    x, _, r, w, positions = _parts(x, weight, positions, eps, norm)
    return _turn(x * r * w, positions, inv_freq, interleaved, 1.0)


def backward(x, weight, positions, inv_freq, dy, eps=1e-6, norm="rms", interleaved=False):
    """(dx, dweight)"""
    x, m, r, w, positions = _parts(x, weight, positions, eps, norm)
    dz = _turn(np.asarray(dy, np.float64), positions, inv_freq, interleaved, -1.0)
    dx = r * w * dz - x * r ** 3 / m * (w * dz * x).sum(-1, keepdims=True)
    return dx, (dz * x * r).sum((0, 1, 2))
