"""GPU checks of what the gated delta rule's results are off by, closer than the
parity tests' norms over all heads and rows.

With bf16 io an output that ends in bf16 is the float32 result rounded once.
Let x be that float32 result, off from the reference by at most t = 6 * 2^-16 +
(N + 128) 2^-24 of the output's root mean square (operands of two bf16 terms,
each off by at most 2^-16, at most six of them on the way, and the float32 sums
of the parity tests).  x and the reference round to different bf16 values only
where a border between two roundings lies between them.  Borders are one step
apart, at least 2^-8 of the value, so among the values of at least half the root
mean square that happens to a share of at most t / (2^-8 / 2) = 2^9 t of them.
A single bf16 operand on the way (2^-8) would make it a third.
"""
import numpy as np
import pytest
import torch

from oracle import delta as od
from state_space_model_mamba_amd import delta
from tests.test_gpu_delta import args, cuda, f64, make, tolerance

pytestmark = pytest.mark.gpu


def rounded_once(got, ref, N, label):
    ref = np.asarray(ref, np.float64)
    want = torch.from_numpy(ref).float().bfloat16()
    big = torch.from_numpy(np.abs(ref) >= 0.5 * np.sqrt((ref * ref).mean()))
    share = (got.cpu() != want)[big].double().mean().item()
    bound = 2.0 ** 9 * (6 * 2.0 ** -16 + (N + 128) * 2.0 ** -24)
    print(f"  {label}: {share:.4f} of {int(big.sum())} values rounded otherwise (bound {bound:.4f})", flush=True)
    assert share <= bound, f"{label}: {share:.4f} > {bound:.4f}"


SHAPES = [(1, 200, 4, 64, 1, 128, None), (1, 500, 8, 64, 2, 64, [100, 1, 64, 335]), (2, 130, 6, 96, 3, 128, None)]


@pytest.mark.parametrize("b,L,H,P,G,N,lengths", SHAPES)
def test_o_is_rounded_once(b, L, H, P, G, N, lengths):
    print(f"[case] o b={b} L={L} H={H} P={P} G={G} N={N}", flush=True)
    d = make(b, L, H, P, G, N, "bf16", seed=31 + L, lengths=lengths, initial=True)
    c = cuda(d)
    o = delta.delta_fwd(*args(c), c["initial_states"], c["seq_idx"], nseqs=d["nseqs"])["o"]
    seq = None if d["seq_idx"] is None else d["seq_idx"].numpy()
    rounded_once(o, od.forward(*[f64(x) for x in args(d)], f64(d["initial_states"]), seq)["o"], N, "o")


@pytest.mark.parametrize("b,L,H,P,G,N,lengths", SHAPES)
def test_gradients_of_rows_are_rounded_once(b, L, H, P, G, N, lengths):
    print(f"[case] gradients b={b} L={L} H={H} P={P} G={G} N={N}", flush=True)
    d = make(b, L, H, P, G, N, "bf16", seed=41 + L, lengths=lengths, initial=True)
    c = cuda(d)
    g = delta.delta_bwd(*args(c), c["do"], c["initial_states"], c["seq_idx"], c["dfin"], nseqs=d["nseqs"])
    seq = None if d["seq_idx"] is None else d["seq_idx"].numpy()
    ref = od.backward(*[f64(x) for x in args(d)], f64(d["do"]), f64(d["initial_states"]), seq, f64(d["dfin"]))
    for k in ("dq", "dk", "dv"):
        rounded_once(g[k], ref[k], N, k)


# decays of a head, the same at every row: from next to none to one that leaves nothing in float32
DECAYS = (0.0, -0.1, -1.0, -4.0, -8.0, -12.0, -30.0, -80.0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("initial", [False, True])
def test_dg_of_every_head_however_strong_its_decay(initial, io):
    """dg_t is exp(g_t) times an inner product of the state before and a gradient after: its error is held against
    each head's own dg, with the parity tests' bound for one head, not against the milder heads beside it."""
    H, N = len(DECAYS), 64
    d = make(1, 200, H, 32, 2, N, io, seed=51, initial=initial)
    d["g"] = torch.tensor(DECAYS).expand(1, 200, H).contiguous()
    c = cuda(d)
    ref = od.backward(*[f64(x) for x in args(d)], f64(d["do"]), f64(d["initial_states"]), None, f64(d["dfin"]))["dg"]
    dg = f64(delta.delta_bwd(*args(c), c["do"], c["initial_states"], None, c["dfin"])["dg"])
    tol = tolerance(torch.float32, d["q"].dtype, N)
    errs = [np.linalg.norm(dg[..., h] - ref[..., h]) / np.linalg.norm(ref[..., h]) for h in range(H)]
    for h in range(H):
        print(f"  {io} g = {DECAYS[h]}: dg {errs[h]:.2e} off (tolerance {tol:.1e})", flush=True)
    assert max(errs) <= tol


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_dg_of_a_dropped_state_is_zero(io):
    d = make(1, 150, 2, 24, 1, 40, io, seed=52, initial=True)
    rows = [0, 17, 64, 65, 149]
    d["g"][0, rows, 0] = -float("inf")
    d["g"][0, rows, 1] = -500.0
    c = cuda(d)
    dg = delta.delta_bwd(*args(c), c["do"], c["initial_states"], None, c["dfin"])["dg"]
    assert bool((dg[0, rows] == 0).all()), dg[0, rows]


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_dg_of_single_rows_among_mild_ones(io):
    """One strong decay here and there: those rows' dg is small beside their neighbours' and still their own."""
    N = 64
    d = make(1, 192, 2, 32, 1, N, io, seed=53, initial=True)
    rows = [5, 63, 64, 100, 191]
    d["g"][0, rows] = -9.0
    c = cuda(d)
    ref = od.backward(*[f64(x) for x in args(d)], f64(d["do"]), f64(d["initial_states"]), None, f64(d["dfin"]))["dg"][0, rows]
    dg = f64(delta.delta_bwd(*args(c), c["do"], c["initial_states"], None, c["dfin"])["dg"])[0, rows]
    err, tol = np.linalg.norm(dg - ref) / np.linalg.norm(ref), tolerance(torch.float32, d["q"].dtype, N)
    print(f"  {io} rows of strong decay: dg {err:.2e} off (tolerance {tol:.1e})", flush=True)
    assert err <= tol


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_dg_is_the_differences(io):
    """dg against central differences of the oracle's loss in single gates, strong ones among them."""
    d = make(1, 70, 1, 8, 1, 16, io, seed=54, initial=True)
    d["g"][0, 40], d["g"][0, 66] = -6.0, -3.0
    c = cuda(d)
    dg = f64(delta.delta_bwd(*args(c), c["do"], c["initial_states"], None, c["dfin"])["dg"])
    x, h0, h = [f64(t) for t in args(d)], f64(d["initial_states"]), 1e-4

    def loss(row, step):
        y = [t.copy() for t in x]
        y[3][0, row, 0] += step
        r = od.forward(*y, h0)
        return (r["o"] * f64(d["do"])).sum() + (r["final_states"] * f64(d["dfin"])).sum()

    for row in (0, 1, 30, 40, 63, 64, 66, 69):
        up, down = loss(row, h), loss(row, -h)
        # truncation h^2 / 6 of third derivatives no larger than the terms of the loss, cancellation 2^-52 |loss| / h
        slack = h * h * max(abs(dg).max(), 1.0) + 2.0 ** -50 * (abs(up) + 1) / h
        assert abs((up - down) / (2 * h) - dg[0, row, 0]) <= slack + 2 * tolerance(torch.float32, d["q"].dtype, 16) * np.abs(dg).max(), row


def test_calls_do_not_share_what_they_return_or_were_given():
    """A result's shape is the caller's own, and a scale given as a tensor counts as it is at the call."""
    d = cuda(make(1, 70, 2, 16, 1, 16, "f32", seed=55))
    want = delta.delta_fwd(*args(d))["o"]
    for call in (lambda: delta.delta_fwd(*args(d)), lambda: delta.delta_bwd(*args(d), d["do"])):
        r = call()
        r["shape"].seqlen, r["shape"].scale = 1, 0.0
        assert call()["shape"].seqlen == 70
        assert torch.equal(delta.delta_fwd(*args(d))["o"], want)
    scale = torch.tensor(0.5)
    one = delta.delta_fwd(*args(d), scale=scale)["o"]
    scale.mul_(2)
    two = delta.delta_fwd(*args(d), scale=scale)["o"]
    assert torch.equal(one, delta.delta_fwd(*args(d), scale=0.5)["o"]) and torch.equal(two, 2 * one)
    leaves = [x.clone().requires_grad_(True) for x in args(d)]
    o, _ = delta.gated_delta_rule(*leaves, scale=scale)
    scale.zero_()
    got = torch.autograd.grad(o, leaves, d["do"])
    ref = delta.delta_bwd(*args(d), d["do"], scale=1.0)
    assert all(torch.equal(a, ref[k]) for a, k in zip(got, ("dq", "dk", "dv", "dg", "dbeta")))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_what_is_added_to_a_state_keeps_float32(io):
    """Every row of a chunk with a key (or query) direction of its own, so a state's columns are single products:
    S[:, n] = beta_n exp(c_last - c_n) v_n, and backwards dS_in[:, n] = scale exp(c_n) dout_n for keys of zero.  With
    |c| <= 2 the exponent's rounding is 2 * 2^-24 of the result, exp and the products' roundings and the operand's three
    terms at most a dozen 2^-24 more: within 2^-20 (two terms would be off by up to 2^-16)."""
    L = N = 64
    d = make(1, L, 2, 32, 1, N, io, seed=56)
    d["g"] = d["g"] * 0.1
    gen = torch.Generator().manual_seed(57)
    ways = torch.eye(N)[torch.randperm(N, generator=gen)].reshape(1, L, 1, N).to(d["k"].dtype)
    c = d["g"].double().cumsum(1)
    assert float(c.abs().max()) <= 2
    at = ways[0, :, 0].argmax(-1)

    def placed(rows):   # (L, H, P): row t in column at[t] of (1, H, P, N)
        S = torch.zeros(1, 2, 32, N, dtype=torch.float64)
        S[0][..., at] = rows.permute(1, 2, 0)
        return S

    def near(got, want):
        got = got.double().cpu()
        assert bool(((got - want).abs() <= 2.0 ** -20 * want.abs()).all()), ((got - want).abs() / want.abs()).max()

    x = cuda(dict(d, q=torch.zeros_like(ways), k=ways))
    near(delta.delta_fwd(*args(x), want_final_states=True)["final_states"],
         placed(((d["beta"].double() * (c[:, -1:] - c).exp())[..., None] * d["v"].double())[0]))
    x = cuda(dict(d, q=ways, k=torch.zeros_like(ways), initial_states=torch.zeros(1, 2, 32, N)))
    near(delta.delta_bwd(*args(x), x["do"], x["initial_states"], scale=0.5)["d_initial_states"],
         placed((0.5 * c.exp()[..., None] * d["do"].double())[0]))
