"""Pins of the fp64 oracles of the block norms and of the gated linear recurrence:
closed forms, torch's own operations in float64 and central differences of every
gradient."""
import numpy as np
import pytest
import torch

from oracle import block_norm as ob
from oracle import recurrence as orc


def rng(seed):
    return np.random.default_rng(seed)


def differences(f, args, grads, seed, h=1e-6, tol=1e-6):
    """Central differences of f along a random direction of each argument, against <gradient, direction>."""
    r = rng(seed)
    for name, g in grads.items():
        d = r.standard_normal(args[name].shape)
        up, down = dict(args, **{name: args[name] + h * d}), dict(args, **{name: args[name] - h * d})
        num, ana = (f(**up) - f(**down)) / (2 * h), float((g * d).sum())
        assert abs(num - ana) <= tol * max(1.0, abs(ana), np.abs(g).max()), (name, num, ana)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_add_norm_gradients_by_differences(norm):
    r = rng(1)
    a = {k: r.standard_normal((2, 3, 10)) for k in ("x", "residual")} | {k: r.standard_normal(10) for k in ("weight", "bias", "scale")}
    dy, dr = r.standard_normal((2, 3, 10)), r.standard_normal((2, 3, 10))

    def loss(**kw):
        y, out = ob.add_norm(**kw, eps=1e-3, norm=norm)
        return float((dy * y).sum() + (dr * out).sum())

    g = ob.add_norm_backward(a["x"], a["residual"], a["weight"], a["scale"], dy, dr, eps=1e-3, norm=norm)
    differences(loss, a, {"x": g["dx"], "residual": g["dresidual"], "weight": g["dweight"], "bias": g["dbias"], "scale": g["dscale"]}, 2)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid", None])
@pytest.mark.parametrize("first", [False, True])
def test_gated_norm_gradients_by_differences(norm, gate, first):
    r = rng(3)
    a = {k: r.standard_normal((2, 3, 12)) for k in ("x", "z")} | {k: r.standard_normal(12) for k in ("weight", "bias", "scale")}
    if gate is None:
        a.pop("z")
    dout, kw = r.standard_normal((2, 3, 12)), dict(groups=3, eps=1e-3, norm=norm, gate=gate or "silu", norm_before_gate=first)
    g = ob.gated_norm_backward(a["x"], a.get("z"), a["weight"], a["bias"], a["scale"], dout, **kw)
    differences(lambda **v: float((dout * ob.gated_norm(**v, **kw)).sum()), a, {k: g["d" + k] for k in a}, 4)


def test_norms_agree_with_torch():
    r = rng(5)
    x, w, b = r.standard_normal((1, 4, 16)), r.standard_normal(16), r.standard_normal(16)
    t = [torch.from_numpy(v) for v in (x, w, b)]
    ref = torch.nn.functional.layer_norm(t[0], (16,), t[1], t[2], 1e-5).numpy()
    np.testing.assert_allclose(ob.add_norm(x, None, w, b, eps=1e-5, norm="layer")[0], ref, rtol=1e-12, atol=1e-12)
    ref = torch.nn.functional.rms_norm(t[0], (16,), t[1], 1e-5).numpy()
    np.testing.assert_allclose(ob.add_norm(x, None, w, eps=1e-5)[0], ref, rtol=1e-12, atol=1e-12)
    z = torch.from_numpy(r.standard_normal((1, 4, 16)))
    act = torch.nn.functional.silu(z)
    ref = torch.nn.functional.rms_norm((t[0] * act).reshape(1, 4, 2, 8), (8,), None, 1e-5).reshape(1, 4, 16) * t[1]
    np.testing.assert_allclose(ob.gated_norm(x, z.numpy(), w, groups=2, eps=1e-5), ref.numpy(), rtol=1e-12, atol=1e-12)


def test_a_constant_row_has_no_layer_norm():
    y, r = ob.add_norm(np.full((1, 1, 8), 3.0), norm="layer")
    assert np.all(y == 0) and np.all(r == 3)


SEQ = np.array([[0, 0, 0, 1, 1, 4, 4], [4, 5, 5, 5, 5, 5, 5]], np.int32)


@pytest.mark.parametrize("gate", ["log", "sigmoid", "decay"])
@pytest.mark.parametrize("scale", ["one", "complement", "unit"])
@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_gradients_by_differences(gate, scale, packed):
    r = rng(7)
    seq = SEQ if packed else None
    n = len(orc.starts_of((2, 7), seq))
    a = {k: r.standard_normal((2, 7, 5)) for k in ("x", "g", "in_gate")} | {"h0": r.standard_normal((n, 5))}
    if gate == "log":
        a["g"] = -np.abs(a["g"]) - 0.1
    if gate == "decay":
        a["decay"] = -np.abs(r.standard_normal(5)) - 0.1
    dy, df, kw = r.standard_normal((2, 7, 5)), r.standard_normal((n, 5)), dict(gate=gate, input_scale=scale)

    def loss(**v):
        o = orc.forward(**v, seq_idx=seq, **kw)
        return float((dy * o["y"]).sum() + (df * o["final_states"]).sum())

    g = orc.backward(a["x"], a["g"], a["in_gate"], a.get("decay"), dy, a["h0"], seq, df, **kw)
    names = {"x": "dx", "g": "dg", "in_gate": "d_in_gate", "h0": "d_initial_states"} | ({"decay": "ddecay"} if gate == "decay" else {})
    differences(loss, a, {k: g[v] for k, v in names.items()}, 8)


def test_recurrence_closed_forms():
    # a = 1/2 and x = 1: h_t = 2 - 2^-t with m = 1, 1 - 2^-(t+1) with m = 1 - a
    x, g = np.ones((1, 20, 1)), np.zeros((1, 20, 1))
    t = np.arange(20.0)
    np.testing.assert_allclose(orc.forward(x, g)["y"][0, :, 0], 2 - 2.0 ** -t, rtol=1e-14)
    np.testing.assert_allclose(orc.forward(x, g, input_scale="complement")["y"][0, :, 0], 1 - 2.0 ** -(t + 1), rtol=1e-14)
    # a state that decays alone; one that is dropped
    y = orc.forward(np.zeros((1, 3, 1)), np.array([[[-1.0], [-2.0], [-np.inf]]]), h0=np.array([[5.0]]), gate="log")["y"]
    np.testing.assert_allclose(y[0, :, 0], [5 * np.exp(-1), 5 * np.exp(-3), 0], rtol=1e-14)
    # unit inputs of unit variance keep it: m^2 = 1 - a^2
    a = orc._gates(np.full((1, 1), 0.3), np.array([-0.7]), "decay", "unit")
    np.testing.assert_allclose(a[0] ** 2 + a[1] ** 2, 1, rtol=1e-14)


def test_sequences_apart_are_the_sequences_packed():
    r = rng(9)
    x, g, h0 = r.standard_normal((2, 7, 3)), r.standard_normal((2, 7, 3)), r.standard_normal((5, 3))
    o = orc.forward(x, g, h0=h0, seq_idx=SEQ)
    edges = [0, 3, 5, 7, 8, 14]
    assert list(orc.starts_of((2, 7), SEQ)) == edges[:-1]
    flat = lambda t: t.reshape(14, 3)  # noqa: E731
    for s in range(5):
        part = slice(edges[s], edges[s + 1])
        one = orc.forward(flat(x)[None, part], flat(g)[None, part], h0=h0[s:s + 1])
        np.testing.assert_array_equal(flat(o["y"])[part], one["y"][0])
        np.testing.assert_array_equal(o["final_states"][s], one["final_states"][0])


@pytest.mark.parametrize("wrong", ["decay of the next row", "no slope of m", "carry over a start"])
def test_planted_mistakes_are_seen(wrong):
    """The differences above reject gradients with one term wrong."""
    r = rng(11)
    x, g, dy = (r.standard_normal((2, 7, 5)) for _ in range(3))
    kw = dict(input_scale="unit")
    good = orc.backward(x, g, None, None, dy, seq_idx=SEQ, **kw)
    if wrong == "no slope of m":
        bad = orc.backward(x, g, None, None, dy, seq_idx=SEQ)["dg"]
    elif wrong == "carry over a start":
        bad = orc.backward(x, g, None, None, dy, **kw)["dg"]
    else:
        bad = np.roll(good["dg"], 1, axis=1)
    loss = lambda x, g: float((dy * orc.forward(x, g, seq_idx=SEQ, **kw)["y"]).sum())  # noqa: E731
    differences(loss, {"x": x, "g": g}, {"x": good["dx"], "g": good["dg"]}, 12)
    with pytest.raises(AssertionError):
        differences(loss, {"x": x, "g": g}, {"g": bad}, 12)
