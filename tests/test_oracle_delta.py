"""The fp64 oracles of the gated delta rule and of the q/k norm, pinned on the
CPU: a hand-worked pair of steps, the solved form of the recurrence, finite
differences of every input, and closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import delta as od
from oracle import qk_norm as on


def inputs(b=2, L=7, H=4, P=3, G=2, N=5, seed=0):
    rng = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    return dict(q=unit(rng.standard_normal((b, L, G, N))), k=unit(rng.standard_normal((b, L, G, N))),
                v=rng.standard_normal((b, L, H, P)), g=-rng.random((b, L, H)), beta=rng.random((b, L, H)))


def test_two_steps_by_hand():
    # P = 1, N = 2, scale 1, S_0 = (2, 0), decay 1/2 a step
    # t = 1: Sd = (1, 0), k = (1, 1), v = 3: e = 3 - 1 = 2; beta 1/2: S = (1, 0) + 1/2 2 (1, 1) = (2, 1); q = (1, -1): o = 1
    # t = 2: Sd = (1, 1/2), k = (0, 2), v = 0: e = -1; beta 1: S = (1, 1/2) - (0, 2) = (1, -3/2); q = (2, 2): o = -1
    f = lambda *x: np.array(x, np.float64)  # noqa: E731
    q, k = f([1, -1], [2, 2]).reshape(1, 2, 1, 2), f([1, 1], [0, 2]).reshape(1, 2, 1, 2)
    v, beta = f(3, 0).reshape(1, 2, 1, 1), f(0.5, 1).reshape(1, 2, 1)
    g = np.full((1, 2, 1), math.log(0.5))
    r = od.forward(q, k, v, g, beta, f(2, 0).reshape(1, 1, 1, 2), None, 1.0)
    np.testing.assert_allclose(r["o"].ravel(), [1, -1], atol=1e-15)
    np.testing.assert_allclose(r["final_states"].ravel(), [1, -1.5], atol=1e-15)


def test_solved_form():
    # (I + diag(beta) N) u = beta (v - exp(c) S0 k), o = scale (exp(c) S0 q + sum exp(c_i - c_j) q.k u), over the whole sequence
    x = inputs(b=1, L=9, H=2, G=1)
    S0 = np.random.default_rng(3).standard_normal((1, 2, 3, 5))
    ref = od.forward(**x, initial_states=S0, scale=0.7)
    for h in range(2):
        c, q, k, v, be = x["g"][0, :, h].cumsum(), x["q"][0, :, 0], x["k"][0, :, 0], x["v"][0, :, h], x["beta"][0, :, h]
        G = np.tril(np.exp(c[:, None] - c[None, :]))
        A = np.eye(9) + be[:, None] * np.tril(G * (k @ k.T), -1)
        u = np.linalg.solve(A, be[:, None] * (v - np.exp(c)[:, None] * (k @ S0[0, h].T)))
        o = 0.7 * (np.exp(c)[:, None] * (q @ S0[0, h].T) + (G * (q @ k.T)) @ u)
        S = np.exp(c[-1]) * S0[0, h] + (np.exp(c[-1] - c)[:, None] * u).T @ k
        np.testing.assert_allclose(ref["o"][0, :, h], o, rtol=0, atol=1e-13)
        np.testing.assert_allclose(ref["final_states"][0, h], S, rtol=0, atol=1e-13)


@pytest.mark.parametrize("packed", [False, True])
def test_gradients_are_the_differences(packed):
    x = inputs()
    seq = np.array([[0, 0, 1, 1, 1, 0, 0], [4, 4, 4, 4, 4, 4, 5]]) if packed else None
    S = 5 if packed else 2
    rng = np.random.default_rng(1)
    S0, dout, dfin = (rng.standard_normal(s) for s in ((S, 4, 3, 5), (2, 7, 4, 3), (S, 4, 3, 5)))
    assert len(od.sequences(2, 7, seq)) == S
    grads = od.backward(**x, dout=dout, initial_states=S0, seq_idx=seq, d_final_states=dfin)

    def loss(y, s0):
        r = od.forward(**y, initial_states=s0, seq_idx=seq)
        return (r["o"] * dout).sum() + (r["final_states"] * dfin).sum()

    for name in ("q", "k", "v", "g", "beta", "initial_states"):
        arg = S0 if name == "initial_states" else x[name]
        d = rng.standard_normal(arg.shape)
        h = 1e-5
        up, down = ((loss(x, S0 + s * h * d) if name == "initial_states" else loss({**x, name: arg + s * h * d}, S0)) for s in (1, -1))
        got = (grads["d_" + name if name == "initial_states" else "d" + name] * d).sum()
        # central differences in double: truncation h^2 = 1e-10, cancellation 1e-16 / h = 1e-11, of values of order 1 to 100
        assert abs((up - down) / (2 * h) - got) <= 1e-7 * max(1.0, abs(got)), name


def test_drop_of_the_state_and_zero_beta():
    x = inputs(b=1, L=4)
    x["g"][0, 2] = -np.inf
    x["beta"][0, 1] = 0
    S0 = np.ones((1, 4, 3, 5))
    whole = od.forward(**x, initial_states=S0)
    rest = od.forward(**{n: a[:, 2:] for n, a in x.items()})   # nothing before row 2 is left
    np.testing.assert_allclose(whole["o"][:, 2:], rest["o"], atol=1e-15)
    g = od.backward(**x, dout=np.ones((1, 4, 4, 3)), initial_states=S0)
    assert np.all(g["dv"][0, 1] == 0) and np.any(g["dbeta"][0, 1] != 0) and np.all(np.isfinite(g["dg"]))
    assert np.all(g["dg"][0, 2] == 0)


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_norm_against_autograd(norm, interleaved):
    rng = np.random.default_rng(2)
    x, w, dy = rng.standard_normal((2, 3, 2, 10)), rng.standard_normal(10), rng.standard_normal((2, 3, 2, 10))
    pos, freq = rng.integers(0, 100, (2, 3)), rng.random(3)
    xt, wt = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    r = torch.rsqrt((xt * xt).mean(-1, keepdim=True) + 1e-3) if norm == "rms" else torch.rsqrt((xt * xt).sum(-1, keepdim=True) + 1e-3)
    z = xt * r * wt
    t = torch.tensor(pos, dtype=torch.float64)[..., None, None] * torch.tensor(freq)
    a, b = (z[..., 0:6:2], z[..., 1:6:2]) if interleaved else (z[..., :3], z[..., 3:6])
    a, b = a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()
    y = torch.cat([torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1), z[..., 6:]], -1)
    y.backward(torch.tensor(dy))
    np.testing.assert_allclose(on.forward(x, w, pos, freq, 1e-3, norm, interleaved), y.detach().numpy(), atol=1e-13)
    dx, dw = on.backward(x, w, pos, freq, dy, 1e-3, norm, interleaved)
    np.testing.assert_allclose(dx, xt.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, wt.grad.numpy(), atol=1e-12)


def test_qk_norm_closed_forms():
    x = np.array([3.0, 4.0]).reshape(1, 1, 1, 2)
    np.testing.assert_allclose(on.forward(x, eps=0.0, norm="l2").ravel(), [0.6, 0.8])
    np.testing.assert_allclose(on.forward(x, eps=0.0).ravel(), np.array([0.6, 0.8]) * math.sqrt(2))
    # a quarter turn: (a, b) -> (-b, a)
    y = on.forward(x, None, np.array([[1]]), np.array([math.pi / 2]), 0.0, "l2")
    np.testing.assert_allclose(y.ravel(), [-0.8, 0.6], atol=1e-15)
