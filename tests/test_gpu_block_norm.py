"""GPU parity of the norms before and after a block, and of their gradients, with
the fp64 oracle.

Tolerances, on the 2-norm of the difference over that of the terms that are
summed: the float32 arithmetic of a value (the sum of W squares and, in the
backward, of W products, the root, the gate's exponential and reciprocal of an
argument up to 16 and at most sixteen more operations) is off by at most
(2 W + 64) 2^-24; sums over rows add one rounding a row, rows 2^-24; bf16
outputs add their own rounding, 2^-8.  Where a gradient is a difference the
norm of its parts stands in the denominator (`parts`): du = r (d - ...) by r d.
"""
import numpy as np
import pytest
import torch

from oracle import block_norm as ob
from state_space_model_mamba_amd import block_norm as bn

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy() if isinstance(t, torch.Tensor) else t


def near(got, ref, W, label, rows=0, parts=None):
    base = max(np.linalg.norm(ref), 0 if parts is None else np.linalg.norm(parts), 1e-30)
    err = np.linalg.norm(f64(got) - ref) / base
    tol = (2 * W + 64 + rows) * 2.0 ** -24 + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0)
    print(f"  {label}: {err:.2e} (tolerance {tol:.1e})", flush=True)
    assert err <= tol, f"{label}: {err:.3e} > {tol:.3e}"


def make(b, L, D, io, residual=None, weight=True, bias=False, scale=1.0, z=False, seed=0, gain=1.0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    t, rt = IO[io], IO[residual or io]
    d = {"x": (gain * rn(b, L, D)).to(t), "z": rn(b, L, D).mul(2).to(t) if z else None, "residual": (gain * rn(b, L, D)).to(rt) if residual else None,
         "weight": 1 + 0.2 * rn(D) if weight else None, "bias": 0.3 * rn(D) if bias else None,
         "scale": 0.5 + 0.2 * rn(D) if scale == "vector" else scale, "dy": rn(b, L, D).to(t), "dr": rn(b, L, D).to(rt)}
    return d


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def rms_of(v, norm, eps, groups):
    u = v.reshape(v.shape[:-1] + (groups, -1))
    if norm == "layer":
        u = u - u.mean(-1, keepdims=True)
    return (((u * u).mean(-1, keepdims=True) + eps) ** -0.5 * np.ones_like(u)).reshape(v.shape)


def check_add(d, label, norm="rms", eps=1e-6):
    print(f"[case] add_norm {label} {norm}", flush=True)
    c, h = cuda(d), {k: f64(v) for k, v in d.items()}
    y, r = bn.add_norm_fwd(c["x"], c["residual"], c["weight"], c["bias"], c["scale"], eps, norm)
    g = bn.add_norm_bwd(c["x"], c["residual"], c["weight"], c["scale"], c["dy"], c["dr"], eps, norm, want_dbias=True, want_dscale=True,
                        want_dresidual=True, want_dweight=True)
    torch.cuda.synchronize()
    W, rows = d["x"].shape[2], d["x"].shape[0] * d["x"].shape[1]
    ry, rr = ob.add_norm(h["x"], h["residual"], h["weight"], h["bias"], h["scale"], eps, norm)
    near(y, ry, W, "y", parts=None if norm == "rms" else ry * 0 + 1)
    near(r, rr, 8, "r")
    assert r.dtype == (d["x"] if d["residual"] is None else d["residual"]).dtype
    ref = ob.add_norm_backward(h["x"], h["residual"], h["weight"], h["scale"], h["dy"], h["dr"], eps, norm)
    part = rms_of(rr, norm, eps, 1) * h["dy"] * (1 if h["weight"] is None else h["weight"])
    near(g["dx"], ref["dx"], W, "dx", parts=part * h["scale"])
    near(g["dresidual"], ref["dresidual"], W, "dresidual", parts=part)
    for k in ("dweight", "dbias"):
        near(g[k], ref[k], W, k, rows)
    number = 1 if isinstance(d["scale"], torch.Tensor) else d["scale"]   # dscale is then that of a vector of ones beside the number
    near(g["dscale"], number * ref["dscale"], W, "dscale", rows, parts=number * np.sqrt(((part * h["x"]) ** 2).sum((0, 1))))


def check_gated(d, label, norm="rms", eps=1e-6, groups=1, gate="silu", first=False):
    print(f"[case] gated_norm {label} {norm} {gate} groups={groups} first={first}", flush=True)
    c, h = cuda(d), {k: f64(v) for k, v in d.items()}
    kw = dict(groups=groups, eps=eps, norm=norm, gate=gate, norm_before_gate=first)
    out = bn.gated_norm_fwd(c["x"], c["z"], c["weight"], c["bias"], c["residual"], c["scale"], **kw)
    g = bn.gated_norm_bwd(c["x"], c["z"], c["weight"], c["bias"], c["scale"], c["dr"], **kw, want_dweight=True, want_dbias=True, want_dscale=True)
    torch.cuda.synchronize()
    W, rows = d["x"].shape[2] // groups, d["x"].shape[0] * d["x"].shape[1]
    ref = ob.gated_norm(h["x"], h["z"], h["weight"], h["bias"], h["residual"], h["scale"], **kw)
    near(out, ref, W, "out")
    ref = ob.gated_norm_backward(h["x"], h["z"], h["weight"], h["bias"], h["scale"], h["dr"], **kw)
    act, slope = (np.ones_like(h["x"]), None) if h["z"] is None else ob._act(h["z"], gate)
    u = h["x"] * (1 if first else act)
    part = rms_of(u, norm, eps, groups) * h["dr"] * h["scale"] * (act if first else 1) * (1 if h["weight"] is None else h["weight"])
    near(g["dx"], ref["dx"], W, "dx", parts=part * (1 if first else act))
    if h["z"] is None:
        assert g["dz"] is None
    else:
        near(g["dz"], ref["dz"], W, "dz", parts=None if first else part * h["x"] * slope)
    number = 1 if isinstance(d["scale"], torch.Tensor) else d["scale"]
    for k in ("dweight", "dbias", "dscale"):
        near(g[k], ref[k] * (number if k == "dscale" else 1), W, k, rows)


SIZES = [(1, 1, 8), (1, 1, 4096), (2, 3, 16), (3, 50, 64), (1, 7, 136), (2, 33, 512), (1, 40, 520), (1, 9, 1000), (2, 5, 2560), (1, 6, 4104), (1, 5, 8192),
         (1, 3, 16384), (1, 700, 40)]


@pytest.mark.parametrize("io,residual", [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("b,L,D", SIZES)
def test_add_norm(b, L, D, io, residual):
    check_add(make(b, L, D, io, residual, weight=L != 3, bias=bool(D % 16), scale="vector" if L % 2 else 0.7, seed=D + L), f"{io}/{residual} {b}x{L}x{D}",
              norm="layer" if D % 16 or L == 5 else "rms")


@pytest.mark.parametrize("io,residual", [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("b,L,W,groups", [(1, 1, 8, 1), (2, 3, 16, 5), (1, 50, 64, 64), (2, 20, 104, 8), (1, 1, 1024, 8), (1, 33, 512, 3), (1, 9, 1000, 1), (2, 4, 1032, 2),
                                          (1, 3, 4096, 2), (1, 3, 8192, 1), (1, 2, 16384, 1), (1, 600, 128, 1)])
def test_gated_norm(b, L, W, groups, io, residual):
    first, z = bool(L % 2), W != 104
    check_gated(make(b, L, W * groups, io, residual, bias=bool(W % 16) or L == 50, scale="vector" if L == 3 else 1.3, z=z, seed=W + L),
                f"{io}/{residual} {b}x{L}x{groups}x{W}", norm="layer" if L % 4 == 1 else "rms", groups=groups,
                gate="sigmoid" if W % 3 == 1 else "silu", first=first)


@pytest.mark.parametrize("gain", [1e-20, 1e15])
def test_values_far_from_one(gain):
    check_add(make(1, 4, 64, "f32", "f32", seed=1, gain=gain), f"gain {gain}")
    check_gated(make(1, 4, 64, "f32", z=True, seed=2, gain=gain), f"gain {gain}")


def test_gates_at_their_ends():
    # saturated gates keep the small side's bits: sigmoid(-16) and 1 - sigmoid(16)
    d = make(1, 4, 64, "f32", z=True, seed=3)
    d["z"] = torch.linspace(-16, 16, 256).reshape(1, 4, 64).contiguous()
    check_gated(d, "silu to 16", first=True)
    check_gated(d, "sigmoid to 16", first=True, gate="sigmoid")
    c = cuda(d)
    g = bn.gated_norm_bwd(c["x"], c["z"], c["weight"], None, 1.0, c["dr"], gate="sigmoid", norm_before_gate=True)
    ref = ob.gated_norm_backward(*[f64(d[k]) for k in ("x", "z", "weight")], None, 1.0, f64(d["dr"]), gate="sigmoid", norm_before_gate=True)
    far = (d["z"].abs() > 12).numpy()
    assert np.max(np.abs(f64(g["dz"])[far] / ref["dz"][far] - 1)) < (2 * 64 + 64) * 2.0 ** -24


def test_empty_gradients_and_absent_sums():
    d = cuda(make(1, 5, 64, "bf16", "f32", seed=4))
    full = bn.add_norm_bwd(d["x"], d["residual"], d["weight"], 1.0, d["dy"], torch.zeros_like(d["dr"]))
    part = bn.add_norm_bwd(d["x"], d["residual"], d["weight"], 1.0, d["dy"], None)
    assert torch.equal(full["dx"], part["dx"]) and torch.equal(full["dresidual"], part["dresidual"]) and part["dbias"] is None and part["dscale"] is None
    only = bn.add_norm_bwd(d["x"], d["residual"], d["weight"], 0.5, None, d["dr"])
    assert torch.equal(only["dresidual"], d["dr"]) and bool((only["dweight"] == 0).all()) and torch.equal(only["dx"], (0.5 * d["dr"]).bfloat16())
    same = bn.add_norm_bwd(d["x"], d["dr"].bfloat16(), d["weight"], 1.0, d["dy"], None)
    assert same["dresidual"] is same["dx"]


@pytest.mark.parametrize("D,groups", [(64, 4), (2560, 1)])
def test_a_bad_row_stays_alone(D, groups):
    d = cuda(make(1, 9, D, "f32", z=True, seed=5))
    good = bn.gated_norm_fwd(d["x"], d["z"], d["weight"], groups=groups)
    gb = bn.gated_norm_bwd(d["x"], d["z"], d["weight"], None, 1.0, d["dr"], groups=groups)
    d["x"][0, 4, 3] = float("nan")
    bad = bn.gated_norm_fwd(d["x"], d["z"], d["weight"], groups=groups)
    bb = bn.gated_norm_bwd(d["x"], d["z"], d["weight"], None, 1.0, d["dr"], groups=groups)
    keep = [i for i in range(9) if i != 4]
    assert torch.equal(good[:, keep], bad[:, keep]) and torch.equal(gb["dx"][:, keep], bb["dx"][:, keep]) and bool(bad[0, 4, 3].isnan())
    if groups > 1:
        assert torch.equal(good[0, 4, D // groups:], bad[0, 4, D // groups:])


def test_a_row_of_zeros_without_eps_stays_alone():
    # 8 rows of 64 lie in a block that has places for 32: nothing of the places without a row reaches the sums
    d = cuda(make(1, 8, 64, "f32", seed=6))
    g = bn.add_norm_bwd(d["x"], None, d["weight"], 1.0, d["dy"], d["dr"], eps=0.0, want_dbias=True, want_dscale=True)
    assert all(bool(torch.isfinite(g[k]).all()) for k in ("dx", "dweight", "dbias", "dscale"))


def test_slices_of_wider_rows_and_bits_on_repeat():
    d = cuda(make(2, 300, 256, "bf16", z=True, seed=7))
    row = torch.cat([d["z"], d["x"], d["z"]], -1)
    s = dict(d, z=row[..., :256], x=row[..., 256:512])
    first = None
    for t in (d, s, d):
        ws = torch.randint(0, 256, (1 << 22,), dtype=torch.uint8, device="cuda")
        out = [bn.gated_norm_fwd(t["x"], t["z"], t["weight"], groups=2), *bn.add_norm_fwd(t["x"], None, t["weight"])]
        g = bn.gated_norm_bwd(t["x"], t["z"], t["weight"], None, 1.0, d["dr"], groups=2, workspace=ws)
        a = bn.add_norm_bwd(t["x"], None, t["weight"], 1.0, d["dy"], d["dr"], workspace=ws)
        out += [g["dx"], g["dz"], g["dweight"], a["dx"], a["dweight"]]
        first = first or out
        assert all(torch.equal(p, q) for p, q in zip(first, out))


def test_operands_larger_than_the_caches():
    # 16384 x 2048: read past the caches, as a part of its rows is not; rows are alone but for the weight's gradient
    gen = torch.Generator(device="cuda").manual_seed(12)
    x, z, dout = (torch.randn((1, 16384, 2048), generator=gen, device="cuda").bfloat16() for _ in range(3))
    w = 1 + 0.1 * torch.randn((2048,), generator=gen, device="cuda")
    whole = bn.gated_norm_bwd(x, z, w, None, 1.0, dout, groups=2)
    add = bn.add_norm_bwd(x, z, w, 1.0, dout, z)
    sums = [torch.zeros(2048, dtype=torch.float64, device="cuda") for _ in range(2)]
    for r in range(0, 16384, 4096):
        at = slice(r, r + 4096)
        g = bn.gated_norm_bwd(x[:, at], z[:, at], w, None, 1.0, dout[:, at], groups=2)
        a = bn.add_norm_bwd(x[:, at], z[:, at], w, 1.0, dout[:, at], z[:, at])
        assert torch.equal(g["dx"], whole["dx"][:, at]) and torch.equal(g["dz"], whole["dz"][:, at]) and torch.equal(a["dx"], add["dx"][:, at])
        sums[0] += g["dweight"]
        sums[1] += a["dweight"]
    for s, t in zip(sums, (whole["dweight"], add["dweight"])):   # at most 64 rows of a block are added in float32, then rounded
        assert float((t - s).norm() / s.norm()) < 2 * 64 * 2.0 ** -24 * (16384 ** 0.5)


def test_rows_past_32_bits():
    # rows 2^23 elements apart: the last begins past 2^31 elements
    wide = torch.empty((300, 1 << 23), dtype=torch.bfloat16, device="cuda")
    x = wide[None, :, :64]
    x.copy_(torch.randn((1, 300, 64), generator=torch.Generator().manual_seed(8)))
    y, r = bn.add_norm_fwd(x)
    z = bn.add_norm_fwd(x.contiguous())
    assert torch.equal(y, z[0]) and torch.equal(r, z[1])


def test_autograd_matches_the_entry_points_and_a_replayed_graph():
    d = cuda(make(1, 40, 128, "bf16", "f32", bias=True, scale="vector", z=True, seed=9))
    leaves = {k: d[k].clone().requires_grad_(True) for k in ("x", "residual", "weight", "bias", "scale")}
    y, r = bn.add_norm(*leaves.values())
    got = torch.autograd.grad((y, r), list(leaves.values()), (d["dy"], d["dr"]))
    g = bn.add_norm_bwd(d["x"], d["residual"], d["weight"], d["scale"], d["dy"], d["dr"], want_dbias=True)
    assert all(torch.equal(a, g["d" + k]) for a, k in zip(got, leaves))
    leaves["z"] = d["z"].clone().requires_grad_(True)
    order = ("x", "z", "weight", "bias", "residual", "scale")
    out = bn.gated_norm(*[leaves[k] for k in order], groups=4)
    got = torch.autograd.grad(out, [leaves[k] for k in order], d["dr"])
    h = bn.gated_norm_bwd(d["x"], d["z"], d["weight"], d["bias"], d["scale"], d["dr"], groups=4)
    h["dresidual"] = d["dr"]
    assert all(torch.equal(a, h["d" + k]) for a, k in zip(got, order))
    # the weight alone, then nothing of r
    w = torch.autograd.grad(bn.add_norm(d["x"], d["residual"], leaves["weight"])[0], leaves["weight"], d["dy"])[0]
    assert torch.equal(w, bn.add_norm_bwd(d["x"], d["residual"], d["weight"], 1.0, d["dy"], None)["dweight"])
    del y, r, out, got, w
    args = [d[k] for k in ("x", "residual", "weight", "scale")]
    ref = [*bn.add_norm_fwd(d["x"], d["residual"], d["weight"], d["bias"], d["scale"]), g["dx"], g["dresidual"], g["dweight"], h["dx"], h["dz"], h["dweight"]]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        f = bn.add_norm_fwd(d["x"], d["residual"], d["weight"], d["bias"], d["scale"])
        a = bn.add_norm_bwd(*args, d["dy"], d["dr"], want_dbias=True)
        b = bn.gated_norm_bwd(d["x"], d["z"], d["weight"], d["bias"], d["scale"], d["dr"], groups=4)
    outs = [*f, a["dx"], a["dresidual"], a["dweight"], b["dx"], b["dz"], b["dweight"]]
    for turn in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, ref)), turn
        for t in outs:
            t.zero_()


def test_one_tensor_in_two_places_and_a_broadcast_gate():
    d = cuda(make(2, 30, 64, "f32", seed=11))
    x = d["x"].clone().requires_grad_(True)
    got = torch.autograd.grad(bn.add_norm(x, x, d["weight"]), x, (d["dy"], d["dr"]))[0]
    g = bn.add_norm_bwd(d["x"], d["x"], d["weight"], 1.0, d["dy"], d["dr"])
    assert torch.equal(got, g["dx"] + g["dresidual"])
    z = torch.randn((1, 30, 64), device="cuda").expand(2, 30, 64)
    a, b = (bn.gated_norm_bwd(d["x"], t, d["weight"], None, 1.0, d["dr"]) for t in (z, z.contiguous()))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dz"], b["dz"])
    assert torch.equal(bn.gated_norm_fwd(d["x"], z, d["weight"]), bn.gated_norm_fwd(d["x"], z.contiguous(), d["weight"]))


def test_another_stream():
    d = cuda(make(1, 64, 512, "bf16", seed=10))
    ref = bn.add_norm_fwd(d["x"], None, d["weight"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = d["x"].clone()
        y = bn.add_norm_fwd(x, None, d["weight"])
    s.synchronize()
    assert torch.equal(y[0], ref[0])


def test_refusals_on_the_device():
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="norm is one of"):
        bn.add_norm_fwd(x, norm="l2")
    with pytest.raises(ValueError, match="gate is one of"):
        bn.gated_norm_fwd(x, x, gate="relu")
    with pytest.raises(ValueError, match="dtype"):
        bn.add_norm_fwd(x, weight=w.bfloat16())
    with pytest.raises(ValueError, match="dtype"):
        bn.add_norm_fwd(x.float(), residual=x)
    with pytest.raises(ValueError, match="shape"):
        bn.gated_norm_fwd(x, x[..., :32])
    with pytest.raises(ValueError, match="contiguous"):
        bn.add_norm_fwd(x.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="unsupported io dtype"):
        bn.add_norm_fwd(x.half())
    with pytest.raises(ValueError, match="needs dy or dr"):
        bn.add_norm_bwd(x, None, None, 1.0, None, None)
    for call in (lambda: bn.gated_norm_fwd(x, groups=3), lambda: bn.add_norm_fwd(x[..., :20].contiguous()), lambda: bn.add_norm_fwd(x[:, :0])):
        with pytest.raises(Exception, match="shape|-2"):
            call()
