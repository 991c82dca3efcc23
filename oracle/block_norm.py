"""fp64 CPU oracle of the norms before and after a block of include/block_norm.h
(test infrastructure only).

With hat = v r, v = u - mean u (u itself for "rms"), r = (mean v^2 + eps)^-1/2
over each group, the gradient d by hat goes back as

    du = r (d - hat mean(d hat) [- mean d])
"""
from __future__ import annotations

import numpy as np


def _unit(u, norm, eps, groups):
    v = np.asarray(u, np.float64).reshape(u.shape[:-1] + (groups, -1))
    if norm == "layer":
        v = v - v.mean(-1, keepdims=True)
    r = ((v * v).mean(-1, keepdims=True) + eps) ** -0.5
    hat = v * r

    def back(d):
        d = d.reshape(v.shape)
        du = d - hat * (d * hat).mean(-1, keepdims=True)
        if norm == "layer":
            du = du - d.mean(-1, keepdims=True)
        return (r * du).reshape(u.shape)

    return hat.reshape(u.shape), back


def _act(z, gate):
    """(act(z), its derivative)"""
    s = np.where(z < 0, np.exp(np.minimum(z, 0)), 1.0) / (1 + np.exp(-np.abs(z)))
    rest = np.where(z < 0, 1.0, np.exp(-np.maximum(z, 0))) / (1 + np.exp(-np.abs(z)))
    return (z * s, s * (1 + z * rest)) if gate == "silu" else (s, s * rest)


def _or(t, value):
    return value if t is None else t


def add_norm(x, residual=None, weight=None, bias=None, scale=1.0, eps=1e-6, norm="rms"):
    """(y, r)"""
    r = scale * x + _or(residual, 0.0)
    hat, _ = _unit(r, norm, eps, 1)
    return hat * _or(weight, 1.0) + _or(bias, 0.0), r


def add_norm_backward(x, residual, weight, scale, dy, dr, eps=1e-6, norm="rms"):
    """dict of dx, dresidual, dweight, dbias, dscale (the last for a scale by channel)"""
    r = scale * x + _or(residual, 0.0)
    hat, back = _unit(r, norm, eps, 1)
    dy, dr = _or(dy, np.zeros_like(x)), _or(dr, np.zeros_like(x))
    g = dr + back(dy * _or(weight, 1.0))
    return {"dx": g * scale, "dresidual": g, "dweight": (dy * hat).sum((0, 1)), "dbias": dy.sum((0, 1)), "dscale": (g * x).sum((0, 1))}


def gated_norm(x, z=None, weight=None, bias=None, residual=None, scale=1.0, groups=1, eps=1e-6, norm="rms", gate="silu", norm_before_gate=False):
    act = 1.0 if z is None else _act(z, gate)[0]
    before, after = (1.0, act) if norm_before_gate else (act, 1.0)
    hat, _ = _unit(x * before, norm, eps, groups)
    return scale * (hat * _or(weight, 1.0) + _or(bias, 0.0)) * after + _or(residual, 0.0)


def gated_norm_backward(x, z, weight, bias, scale, dout, groups=1, eps=1e-6, norm="rms", gate="silu", norm_before_gate=False):
    """dict of dx, dz, dweight, dbias, dscale"""
    act, slope = (1.0, 0.0) if z is None else _act(z, gate)
    before, after = (1.0, act) if norm_before_gate else (act, 1.0)
    hat, back = _unit(x * before, norm, eps, groups)
    n = hat * _or(weight, 1.0) + _or(bias, 0.0)
    dn = dout * scale * after
    du = back(dn * _or(weight, 1.0))
    return {"dx": du * before, "dz": None if z is None else (dout * scale * n if norm_before_gate else du * x) * slope,
            "dweight": (dn * hat).sum((0, 1)), "dbias": dn.sum((0, 1)), "dscale": (dout * n * after).sum((0, 1))}
