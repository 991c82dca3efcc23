"""The norms of include/block_norm.h in float64 with a bound, element by element, of what their float32 arithmetic may be
off by (test infrastructure only; torch, on any device).

Every value carries the bound along: a rounding adds U = 2^-24 of the result, an operation hands on its operands' bounds
times its derivatives.  What the kernels do is counted from above:

    a sum of W            each term passes at most min(W, 16 + 6 + 16) additions: a lane's values, the lanes, the waves
    a mean                the sum, 1 / W and the product: two roundings more
    1 / sqrt(q)           a root and a reciprocal of an ulp each: 4 U
    exp(-|z|)             (2 + 2 |z|) U; 1 / (1 + e): 3 U and e / (1 + e) of that; below 2^-126 nothing is left
    alpha, eps, scale     read in float32: a rounding each
    a sum over rows       each term passes at most `rows` additions, and the result is rounded
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


class Val:
    def __init__(self, v, e=None):
        self.v = v.double() if isinstance(v, torch.Tensor) else torch.tensor(float(v), dtype=torch.float64)
        self.e = torch.zeros_like(self.v) if e is None else e

    def to(self, device):
        return Val(self.v.to(device), self.e.to(device))

    def __add__(self, o):
        v = self.v + o.v
        return Val(v, self.e + o.e + U * v.abs())

    def __sub__(self, o):
        v = self.v - o.v
        return Val(v, self.e + o.e + U * v.abs())

    def __mul__(self, o):
        v = self.v * o.v
        return Val(v, self.e * o.v.abs() + o.e * self.v.abs() + self.e * o.e + U * v.abs())

    def split(self, groups):
        return Val(self.v.unflatten(-1, (groups, -1)), self.e.unflatten(-1, (groups, -1)))

    def join(self):
        return Val(self.v.flatten(-2), self.e.flatten(-2))

    def mean(self):
        """Over the last axis."""
        W = self.v.shape[-1]
        v = self.v.mean(-1, keepdim=True)
        return Val(v, self.e.mean(-1, keepdim=True) + min(W, 38) * U * (self.v.abs() + self.e).mean(-1, keepdim=True) + 2 * U * v.abs())

    def rsqrt(self):
        v = self.v ** -0.5
        # of the slope at the bound's far end
        return Val(v, 0.5 * self.e * (self.v - self.e).clamp(min=1e-300) ** -1.5 + 4 * U * v)

    def rows(self, n):
        """Over all but the last axis, a term passing n additions."""
        axes = tuple(range(self.v.ndim - 1))
        v = self.v.sum(axes)
        return Val(v, self.e.sum(axes) + n * U * (self.v.abs() + self.e).sum(axes) + U * v.abs())


def number(a, device):
    return Val(a, torch.tensor(U * abs(float(a)), dtype=torch.float64)).to(device)


def _factor(scale, device):
    """alpha * scale, as the kernels form it"""
    return Val(scale) if isinstance(scale, torch.Tensor) else number(scale, device)


def _gate(z, gate):
    """(act(z), its derivative)"""
    z = z.double()
    e = torch.exp(-z.abs())
    rel = (2 + 2 * z.abs()) * U
    big, small = 1 / (1 + e), e / (1 + e)
    big, small = Val(big, big * (small * rel + 3 * U)), Val(small, small * (rel + rel * small + 4 * U) + TINY)
    neg = z < 0
    pick = lambda a, b: Val(torch.where(neg, a.v, b.v), torch.where(neg, a.e, b.e))  # noqa: E731
    s, rest = pick(small, big), pick(big, small)
    if gate == "sigmoid":
        return s, s * rest
    z = Val(z)
    one = Val(torch.ones_like(z.v))
    return z * s, s * (z * rest + one)


def _unit(u, norm, eps):
    """(v, 1 / sqrt(mean v^2 + eps)) over the last axis"""
    v = u - u.mean() if norm == "layer" else u
    return v, ((v * v).mean() + number(eps, v.v.device)).rsqrt()


def _back(v, rho, d, norm):
    dot = (d * v).mean() * rho * rho
    inner = d - v * dot
    return rho * (inner - d.mean()) if norm == "layer" else rho * inner


def add_norm(x, residual=None, weight=None, bias=None, scale=1.0, eps=1e-6, norm="rms"):
    """(y, r)"""
    r = _factor(scale, x.device) * Val(x)
    if residual is not None:
        r = r + Val(residual)
    v, rho = _unit(r, norm, eps)
    y = v * rho
    if weight is not None:
        y = y * Val(weight)
    return (y if bias is None else y + Val(bias)), r


def add_norm_backward(x, residual, weight, scale, dy, dr, rows, eps=1e-6, norm="rms"):
    """dict of dx, dresidual, dweight, dbias, dscale (beside a number the scale counts as a vector of ones)"""
    s, xv, dyv = _factor(scale, x.device), Val(x), Val(dy)
    r = s * xv
    if residual is not None:
        r = r + Val(residual)
    v, rho = _unit(r, norm, eps)
    d = dyv if weight is None else dyv * Val(weight)
    g = Val(dr) + _back(v, rho, d, norm)
    ds = (g * xv).rows(rows)
    return {"dx": g * s, "dresidual": g, "dweight": (dyv * (v * rho)).rows(rows), "dbias": dyv.rows(rows),
            "dscale": ds if isinstance(scale, torch.Tensor) else ds * s}


def _gated(x, z, groups, eps, norm, gate, first):
    xs = Val(x).split(groups)
    act, slope = (None, None) if z is None else (t.split(groups) for t in _gate(z, gate))
    v, rho = _unit(xs if act is None or first else xs * act, norm, eps)
    return xs, act, slope, v, rho


def gated_norm(x, z=None, weight=None, bias=None, residual=None, scale=1.0, groups=1, eps=1e-6, norm="rms", gate="silu", norm_before_gate=False):
    _, act, _, v, rho = _gated(x, z, groups, eps, norm, gate, norm_before_gate)
    n = v * rho
    if weight is not None:
        n = n * Val(weight).split(groups)
    if bias is not None:
        n = n + Val(bias).split(groups)
    if act is not None and norm_before_gate:
        n = n * act
    n = n.join() * _factor(scale, x.device)
    return n if residual is None else n + Val(residual)


def gated_norm_backward(x, z, weight, bias, scale, dout, rows, groups=1, eps=1e-6, norm="rms", gate="silu", norm_before_gate=False):
    """dict of dx, dz, dweight, dbias, dscale"""
    xs, act, slope, v, rho = _gated(x, z, groups, eps, norm, gate, norm_before_gate)
    after = act if norm_before_gate else None
    s = _factor(scale, x.device)
    do = Val(dout).split(groups)
    ds = do * (s.split(groups) if isinstance(scale, torch.Tensor) else s)
    dn = ds if after is None else ds * after
    hat = v * rho
    n, d = hat, dn
    if weight is not None:
        w = Val(weight).split(groups)
        n, d = n * w, dn * w
    if bias is not None:
        n = n + Val(bias).split(groups)
    du = _back(v, rho, d, norm)
    dx = du if act is None or norm_before_gate else du * act
    dz = None if z is None else ((ds * n if norm_before_gate else du * xs) * slope).join()
    gs = do * n if after is None else do * n * after
    gs = gs.join().rows(rows)
    return {"dx": dx.join(), "dz": dz, "dweight": (dn * hat).join().rows(rows), "dbias": dn.join().rows(rows),
            "dscale": gs if isinstance(scale, torch.Tensor) else gs * s}
