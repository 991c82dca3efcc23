"""GPU parity of the gated delta rule (whole sequences, gradients, few tokens on
a pool of states) with the fp64 oracle, and its behaviour at the borders.

Tolerances, on the 2-norm of the difference over the 2-norm of the result.
A rounding to bf16 is off by at most 2^-8 of the value.
  * f32 io: a value is reached over at most N + 2 * 64 products and sums in
    float32, each off by 2^-24: (N + 128) 2^-24.
  * bf16 io, bf16 outputs: the output's own rounding and at most three single
    bf16 operands on the way (a state, a correction u, a score): 4 * 2^-8.
  * bf16 io, float32 outputs: operands of two bf16 terms, each off by at most
    2^-16; at most six of them on the way (S, r, T', u, and back dS, du):
    6 * 2^-16, and the float32 part above.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import conv1d as oc
from oracle import delta as od
from oracle import qk_norm as on
from state_space_model_mamba_amd import conv1d, delta, qk_norm, ssd
from state_space_model_mamba_amd.workloads import seq_idx_from_lengths

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "d_initial_states")


def tolerance(dtype, io, N):
    exact = (N + 128) * 2.0 ** -24
    if io == torch.float32:
        return exact
    return 4 * 2.0 ** -8 if dtype == torch.bfloat16 else 6 * 2.0 ** -16 + exact


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(b, L, H, P, G, N, io="bf16", seed=0, lengths=None, initial=False, strong=False, gain=1.0):
    """CPU tensors; ``strong``: decays from none to nearly all of the state."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    unit = lambda x: x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)  # noqa: E731
    t = IO[io]
    d = {"q": unit(rn(b, L, G, N)).to(t), "k": unit(rn(b, L, G, N)).to(t), "v": (gain * rn(b, L, H, P)).to(t),
         "g": -(torch.exp(6 * torch.rand(b, L, H, generator=gen) - 4) if strong else 0.2 * torch.rand(b, L, H, generator=gen)),
         "beta": torch.sigmoid(rn(b, L, H)), "seq_idx": None, "initial_states": None}
    S = b
    if lengths is not None:
        d["seq_idx"] = seq_idx_from_lengths(lengths)
        S = len(lengths)
    d["nseqs"] = S
    if initial:
        d["initial_states"] = 0.3 * rn(S, H, P, N)
    d["do"], d["dfin"] = rn(b, L, H, P).to(t), rn(S, H, P, N)
    return d


def cuda(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def args(d):
    return d["q"], d["k"], d["v"], d["g"], d["beta"]


def near(got, ref, io, N, label, size=None):
    ref = np.asarray(ref, np.float64)
    assert tuple(got.shape) == ref.shape, label
    err = np.linalg.norm(f64(got) - ref) / max(np.linalg.norm(ref if size is None else size), 1e-30)
    tol = tolerance(got.dtype, io, N)
    print(f"  {label}: {err:.2e} (tolerance {tol:.1e})", flush=True)
    assert err <= tol, f"{label}: {err:.3e} > {tol:.3e}"


def dg_terms(d, ref, gref):
    """dg is taken as phi - sum over the chunk's rows i < t of (dout_i . o_i - dv_i . v_i) with phi the dg of the
    chunk's first row, so a relative error of every term of at most x leaves dg off by at most x times the sum of
    the terms' magnitudes, however small dg itself comes out.  That sum, for one sequence a batch row."""
    t = np.abs((f64(d["do"]) * ref["o"]).sum(-1)) + np.abs((gref["dv"] * f64(d["v"])).sum(-1))
    size = np.zeros_like(t)
    for r in range(0, t.shape[1], 64):
        part = t[:, r:r + 64].cumsum(1)
        size[:, r:r + 64] = np.abs(gref["dg"][:, r:r + 1]) + part - t[:, r:r + 64]
    return size


def check(d, label, dfinal=True, scale=None, cancels=False):
    print(f"[case] {label}", flush=True)
    c, io, N = cuda(d), d["q"].dtype, d["q"].shape[3]
    more = dict(scale=scale, nseqs=d["nseqs"])
    r = delta.delta_fwd(*args(c), c["initial_states"], c["seq_idx"], want_final_states=True, **more)
    dfin = c["dfin"] if dfinal else None
    g = delta.delta_bwd(*args(c), c["do"], c["initial_states"], c["seq_idx"], dfin, **more)
    torch.cuda.synchronize()
    n = [f64(x) for x in args(d)]
    seq = None if d["seq_idx"] is None else d["seq_idx"].numpy()
    ref = od.forward(*n, f64(d["initial_states"]), seq, scale)
    gref = od.backward(*n, f64(d["do"]), f64(d["initial_states"]), seq, f64(d["dfin"]) if dfinal else None, scale)
    near(r["o"], ref["o"], io, N, "o")
    near(r["final_states"], ref["final_states"], io, N, "final_states")
    for k in GRADS:
        near(g[k], gref[k], io, N, k, dg_terms(d, ref, gref) if cancels and k == "dg" else None)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("b,L,H,P,G,N", [
    (1, 1, 1, 8, 1, 8), (2, 2, 2, 16, 2, 16), (1, 63, 2, 24, 1, 40), (2, 64, 4, 64, 2, 64), (1, 65, 3, 72, 3, 72), (1, 130, 2, 136, 1, 128),
    (3, 200, 6, 32, 2, 96)])
def test_shapes(b, L, H, P, G, N, io):
    check(make(b, L, H, P, G, N, io, seed=L, initial=b == 2), f"{io} b={b} L={L} H={H} P={P} G={G} N={N}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_packed_sequences(io):
    # lengths of one, starts on and next to the chunks' borders, a long one
    lengths = [1, 1, 62, 64, 65, 1, 127, 3, 200, 128]
    check(make(1, sum(lengths), 4, 40, 2, 48, io, seed=5, lengths=lengths, initial=True), f"{io} packed")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H", [3, 8, 21])
def test_heads_of_one_group_in_parts(H, io):
    # one group and few chunks: its heads go in parts of one or more, the last part short
    check(make(1, 100, H, 16, 1, 72, io, seed=22 + H), f"{io} {H} heads of one group")
    check(make(1, 64 * 60 + 1, H, 8, 1, 8, io, seed=23), f"{io} {H} heads of one group, 61 chunks")


def test_more_sequences_than_a_block_ranks():
    lengths = [1 + i % 3 for i in range(1100)]
    check(make(1, sum(lengths), 1, 8, 1, 8, "f32", seed=21, lengths=lengths, initial=True), "1100 sequences")


def test_packed_rows_of_a_batch_with_recurring_ids():
    d = make(2, 90, 2, 16, 1, 16, "f32", seed=6)
    ids = torch.zeros(2, 90, dtype=torch.int32)
    ids[0, 30:70], ids[1, 1:], ids[1, 88:] = 7, -3, 0
    S = len(od.sequences(2, 90, ids.numpy()))
    assert S == 6
    gen = torch.Generator().manual_seed(1)
    d.update(seq_idx=ids, nseqs=S, initial_states=torch.randn(S, 2, 16, 16, generator=gen), dfin=torch.randn(S, 2, 16, 16, generator=gen))
    check(d, "recurring ids over two rows")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gates_at_their_ends(io):
    d = make(1, 150, 3, 32, 1, 64, io, seed=7, initial=True, strong=True)
    d["g"][0, 10, 0] = -float("inf")
    d["g"][0, 64, 1] = -500.0
    d["g"][0, 100:110, 2] = 0.0
    d["beta"][0, 20:40] = 0.0
    d["beta"][0, 50:60] = 1.0
    check(d, f"{io} decays of nothing and everything, beta 0 and 1")


def test_one_key_for_all_rows():
    # the same key at every row, beta near one: N is dense, T' alternates, and dv undoes most of what later rows say:
    # dg is some four hundred times smaller than the terms whose difference it is
    d = make(1, 130, 2, 32, 1, 32, "f32", seed=8)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 0.9
    check(d, "one key", scale=0.5, cancels=True)


@pytest.mark.parametrize("gain", [1e-12, 1e12])
def test_values_far_from_one(gain):
    # o, the states and dbeta, dg are linear in v: nothing in between leaves the range
    d = make(1, 70, 2, 16, 1, 32, "bf16", seed=9, gain=gain)
    d["dfin"] = torch.zeros_like(d["dfin"])
    check(d, f"gain {gain}", dfinal=False)


def test_without_final_gradient_and_many_chunks():
    check(make(1, 1500, 2, 64, 1, 128, "bf16", seed=10, strong=True), "1500 rows", dfinal=False)


def test_inputs_as_slices_of_wider_rows():
    d = cuda(make(2, 90, 4, 16, 2, 24, "bf16", seed=11))
    row = torch.cat([d["v"].flatten(2), d["k"].flatten(2), d["q"].flatten(2), torch.randn(2, 90, 8, device="cuda").bfloat16()], -1)
    s = dict(d, v=row[..., :64].unflatten(-1, (4, 16)), k=row[..., 64:112].unflatten(-1, (2, 24)), q=row[..., 112:160].unflatten(-1, (2, 24)))
    a, b = delta.delta_fwd(*args(d), want_final_states=True), delta.delta_fwd(*args(s), want_final_states=True)
    ga, gb = delta.delta_bwd(*args(d), d["do"]), delta.delta_bwd(*args(s), d["do"])
    wide = dict(d, k=d["k"][:1].expand(2, 90, 2, 24))   # one batch row's keys for both
    c = delta.delta_fwd(*args(wide))
    e = delta.delta_fwd(*args(dict(d, k=wide["k"].contiguous())))
    torch.cuda.synchronize()
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["final_states"], b["final_states"]) and torch.equal(c["o"], e["o"])
    for k in GRADS:
        assert torch.equal(ga[k], gb[k]), k


def test_bitwise_repeatable_with_garbage_workspace():
    d = cuda(make(1, 777, 8, 72, 2, 128, "bf16", seed=12, lengths=[300, 77, 400], initial=True))
    more = dict(nseqs=3)
    first = None
    for i in range(3):
        gen = torch.Generator(device="cuda").manual_seed(i)
        r = delta.delta_fwd(*args(d), d["initial_states"], d["seq_idx"], want_final_states=True, **more)
        ws = torch.randint(0, 256, (r["workspace"].numel(),), dtype=torch.uint8, device="cuda", generator=gen)
        r = delta.delta_fwd(*args(d), d["initial_states"], d["seq_idx"], want_final_states=True, workspace=ws, **more)
        g = delta.delta_bwd(*args(d), d["do"], d["initial_states"], d["seq_idx"], d["dfin"], **more)
        ws = torch.randint(0, 256, (g["workspace"].numel(),), dtype=torch.uint8, device="cuda", generator=gen)
        g = delta.delta_bwd(*args(d), d["do"], d["initial_states"], d["seq_idx"], d["dfin"], workspace=ws, **more)
        torch.cuda.synchronize()
        bits = [x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32).clone() for x in
                [r["o"], r["final_states"]] + [g[k] for k in GRADS]]
        first = first or bits
        assert all(torch.equal(a, b) for a, b in zip(first, bits))


@pytest.mark.parametrize("H,P,G,N", [(128, 64, 8, 128), (64, 128, 64, 128), (160, 32, 4, 64)])
def test_bits_on_repeat_of_many_chunks(H, P, G, N):
    """Thousands of chunk and head blocks, each the same bits every time (waves of a block share LDS throughout)."""
    d = cuda(make(1, 2048, H, P, G, N, "bf16", seed=20))
    first = None
    for _ in range(6):
        r, g = delta.delta_fwd(*args(d), want_final_states=True), delta.delta_bwd(*args(d), d["do"])
        out = [r["o"], r["final_states"]] + [g[k] for k in GRADS]
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_rows_past_the_last_sequence_stay_as_they_were():
    d = cuda(make(1, 100, 2, 16, 1, 16, "f32", seed=13, lengths=[40, 60]))
    s = delta.make_shape(1, 100, 2, 16, 1, 16, 1, ssd.SSD_IO_F32)   # one sequence of the two
    o = torch.full((1, 100, 2, 16), 7.0, device="cuda")
    ws = torch.empty(delta.workspace_size(s), dtype=torch.uint8, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = delta.load_library().delta_fwd(ctypes.byref(s), *[p(x) for x in args(d)], None, p(d["seq_idx"]), p(o), None, p(ws), ws.numel(),
                                        torch.cuda.current_stream().cuda_stream)
    ref = delta.delta_fwd(*args(d), None, d["seq_idx"], nseqs=2)
    more = delta.delta_fwd(*args(d), None, d["seq_idx"], nseqs=4, want_final_states=True)   # two sequences that are not there
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(o[:, :40], ref["o"][:, :40]) and bool((o[:, 40:] == 7.0).all())
    assert torch.equal(more["o"], ref["o"]) and bool((more["final_states"][2:] == 0).all())


def test_autograd_from_both_outputs():
    d = cuda(make(1, 100, 4, 16, 2, 32, "f32", seed=14, lengths=[30, 70], initial=True))
    leaves = [x.clone().requires_grad_(True) for x in (*args(d), d["initial_states"])]
    o, fin = delta.gated_delta_rule(*leaves, seq_idx=d["seq_idx"])
    torch.autograd.backward([o, fin], [d["do"], d["dfin"]])
    g = delta.delta_bwd(*args(d), d["do"], d["initial_states"], d["seq_idx"], d["dfin"])
    for leaf, k in zip(leaves, GRADS):
        assert torch.equal(leaf.grad, g[k]), k
    o, fin = delta.gated_delta_rule(*leaves, seq_idx=d["seq_idx"])
    got = torch.autograd.grad(fin, leaves[1:], d["dfin"])   # nothing from o
    z = delta.delta_bwd(*args(d), torch.zeros_like(d["do"]), d["initial_states"], d["seq_idx"], d["dfin"])
    for a, k in zip(got, GRADS[1:]):
        assert torch.equal(a, z[k]), k


def test_gradients_that_start_anywhere():
    d = cuda(make(1, 70, 2, 8, 1, 16, "bf16", seed=23))
    leaves = [x.clone().requires_grad_(True) for x in args(d)]
    o, fin = delta.gated_delta_rule(*leaves)
    od, fd = torch.zeros(d["do"].numel() + 1).bfloat16().cuda(), torch.zeros(d["dfin"].numel() + 1).cuda()
    od[1:], fd[1:] = d["do"].flatten(), d["dfin"].flatten()
    got = torch.autograd.grad((o, fin), leaves, (od[1:].view(o.shape), fd[1:].view(fin.shape)))
    g = delta.delta_bwd(*args(d), d["do"], d_final_states=d["dfin"])
    for a, k in zip(got, GRADS):
        assert torch.equal(a, g[k]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_value_that_is_no_number_stays_in_its_sequence(value, io):
    """The middle sequences of a packed batch (one inside a chunk, one of several chunks) full of it."""
    lengths = [70, 9, 1, 150, 30]
    d = cuda(make(1, sum(lengths), 4, 24, 2, 40, io, seed=24, lengths=lengths, initial=True))
    bad = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    for k in ("q", "k", "v", "beta", "do"):
        bad[k][:, 70:79] = value
        bad[k][:, 80:230] = value
    clean = torch.ones(sum(lengths), dtype=torch.bool)
    clean[70:79] = clean[80:230] = False
    kept = [0, 2, 4]
    run = lambda x: (delta.delta_fwd(*args(x), x["initial_states"], x["seq_idx"], want_final_states=True),  # noqa: E731
                     delta.delta_bwd(*args(x), x["do"], x["initial_states"], x["seq_idx"], x["dfin"]))
    (f, g), (bf, bg) = run(d), run(bad)
    rows = clean.cuda()
    for k, a, b in [("o", f["o"], bf["o"])] + [(k, g[k], bg[k]) for k in ("dq", "dk", "dv", "dg", "dbeta")]:
        assert torch.equal(a[:, rows], b[:, rows]), k
    assert torch.equal(f["final_states"][kept], bf["final_states"][kept])
    assert torch.equal(g["d_initial_states"][kept], bg["d_initial_states"][kept])
    assert not torch.isfinite(bf["o"][:, ~rows].float()).all()


def test_step_marks_the_states_as_changed():
    d = cuda(make(1, 1, 2, 8, 1, 16, "bf16", seed=25))
    states = torch.zeros(1, 2, 8, 16, device="cuda")
    w = torch.ones(1, device="cuda", requires_grad=True)
    y = (w * states).sum()   # its backward reads states
    delta.delta_step(*args(d), states)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():
        delta.delta_step(*args(d), torch.zeros(1, 2, 8, 16, device="cuda"))


def test_another_stream_and_replayed_graphs_that_share_a_workspace():
    a, b = cuda(make(1, 200, 4, 64, 1, 128, "bf16", seed=15)), cuda(make(1, 200, 4, 64, 1, 128, "bf16", seed=16))
    eager = [(delta.delta_fwd(*args(x))["o"], delta.delta_bwd(*args(x), x["do"])) for x in (a, b)]
    ws = torch.empty(eager[0][1]["workspace"].numel(), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = delta.delta_fwd(*args(a), workspace=ws)["o"]
        delta.delta_bwd(*args(a), a["do"], workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(o, eager[0][0])
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = delta.delta_fwd(*args(x), workspace=ws)["o"]
            r = delta.delta_bwd(*args(x), x["do"], workspace=ws)
        graphs.append((g, o, r))
    for turn in range(3):
        for (g, o, r), (eo, er) in zip(graphs, eager):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, eo), turn
            for k in ("dq", "dk", "dv", "dg", "dbeta"):
                assert torch.equal(r[k], er[k]), (turn, k)
            ws.fill_(turn + 3)   # eager work between the replays


# ---------------------------------------------------------------------------------------------
# few tokens on a pool of states
# ---------------------------------------------------------------------------------------------
def step_check(d, states, index, label, scale=None):
    print(f"[case] {label}", flush=True)
    io, N = d["q"].dtype, d["q"].shape[3]
    ref_o, ref_s = od.step(*[f64(x) for x in args(d)], f64(states), None if index is None else index.numpy(), scale)
    got_s = states.cuda()
    o = delta.delta_step(*[x.cuda() for x in args(d)], got_s, None if index is None else index.cuda(), scale)
    torch.cuda.synchronize()
    # the state is float32 throughout; o is rounded once
    exact = (N + 64) * 2.0 ** -24 * d["q"].shape[1]
    assert np.linalg.norm(f64(got_s) - ref_s) <= exact * np.linalg.norm(ref_s), label
    assert np.linalg.norm(f64(o) - ref_o) <= (exact + (2.0 ** -8 if io == torch.bfloat16 else 0)) * np.linalg.norm(ref_o), label
    return o, got_s


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("b,T,H,P,G,N,slots", [
    (1, 1, 1, 8, 1, 8, 1), (3, 1, 4, 16, 2, 40, 5), (2, 3, 6, 72, 3, 96, 2), (5, 1, 2, 136, 1, 128, 9), (1, 64, 2, 24, 1, 64, 3),
    (70, 2, 2, 8, 1, 16, 100)])
def test_step_shapes(b, T, H, P, G, N, slots, io):
    d = make(b, T, H, P, G, N, io, seed=b + T, strong=True)
    gen = torch.Generator().manual_seed(b)
    index = torch.randperm(slots, generator=gen)[:b].int() if slots > b else None
    step_check(d, torch.randn(slots, H, P, N, generator=gen), index, f"step {io} b={b} T={T} H={H} P={P} G={G} N={N}", scale=0.3)


def test_step_empty_rows_and_rows_that_share_a_state():
    b = 150
    d = make(b, 2, 2, 24, 1, 32, "f32", seed=3)
    gen = torch.Generator().manual_seed(4)
    states = torch.randn(40, 2, 24, 32, generator=gen)
    index = torch.randint(-2, 42, (b,), generator=gen).int()   # empty rows, rows past the pool, states named many times
    index[0], index[63], index[64], index[149] = 5, 5, 5, 5
    o, got = step_check(d, states, index, "step shared")
    empty = (index < 0) | (index >= 40)
    assert bool((o.cpu()[empty] == 0).all())
    unused = torch.ones(40, dtype=torch.bool)
    unused[index[~empty].long()] = False
    assert torch.equal(got.cpu()[unused], states[unused])


def test_step_keeps_a_dropped_state_finite():
    d = make(2, 1, 1, 8, 1, 8, "f32", seed=5)
    d["g"][0] = -float("inf")
    step_check(d, torch.randn(2, 1, 8, 8, generator=torch.Generator().manual_seed(1)), None, "step drop")


def test_prefill_then_steps_is_the_whole_sequence():
    d = make(2, 140, 4, 64, 2, 128, "bf16", seed=17)
    c = cuda(d)
    cut = lambda a, z: [x[:, a:z].contiguous() for x in args(c)]  # noqa: E731
    whole = delta.delta_fwd(*args(c), want_final_states=True)
    r = delta.delta_fwd(*cut(0, 131), want_final_states=True)
    states, outs = r["final_states"], [r["o"]]
    for t, n in ((131, 1), (132, 5), (137, 3)):
        outs.append(delta.delta_step(*cut(t, t + n), states))
    torch.cuda.synchronize()
    ref = od.forward(*[f64(x) for x in args(d)])
    near(torch.cat(outs, 1), ref["o"], torch.bfloat16, 128, "o")
    near(states, ref["final_states"], torch.bfloat16, 128, "states")
    near(whole["final_states"], ref["final_states"], torch.bfloat16, 128, "whole")


def test_step_in_a_replayed_graph():
    d = cuda(make(3, 1, 4, 64, 2, 128, "bf16", seed=18))
    start = torch.randn(6, 4, 64, 128, device="cuda")
    index = torch.tensor([4, -1, 2], dtype=torch.int32, device="cuda")
    eager, outs = start.clone(), []
    for _ in range(3):
        outs.append(delta.delta_step(*args(d), eager, index))
    states = start.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        o = delta.delta_step(*args(d), states, index)
    states.copy_(start)
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, outs[i]), i
    assert torch.equal(states, eager)


# ---------------------------------------------------------------------------------------------
# a layer's run of them together
# ---------------------------------------------------------------------------------------------
def test_conv_norm_and_delta_rule_as_a_layer():
    """causal conv1d -> slices -> q/k norm with rotation -> gated delta rule, forward and gradients, packed."""
    H, P, G, N, lengths = 4, 16, 2, 32, [50, 1, 79]
    L, C = sum(lengths), 4 * 16 + 2 * 2 * 32
    gen = torch.Generator().manual_seed(19)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, w, bias, do = rn(1, L, C), rn(C, 4) / 2, rn(C) / 2, rn(1, L, H, P)
    g, beta = -0.2 * torch.rand(1, L, H, generator=gen), torch.sigmoid(rn(1, L, H))
    wq, wk = 1 + 0.1 * rn(N), 1 + 0.1 * rn(N)
    freq = (1000.0 ** (-torch.arange(0, 16, 2).double() / 16)).float()
    seq = seq_idx_from_lengths(lengths)
    pos = torch.cat([torch.arange(n) for n in lengths]).int()[None].contiguous()
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, bias, g, beta, wq, wk)]
    lx, lw, lb, lg, lbe, lwq, lwk = leaves
    y = conv1d.causal_conv1d(lx, lw, lb, seq.cuda(), "silu")
    v = y[..., :64].unflatten(-1, (H, P))
    k = y[..., 64:128].unflatten(-1, (G, N))
    q = y[..., 128:].unflatten(-1, (G, N))
    q, k = qk_norm.qk_norm_rope(q, k, lwq, lwk, pos.cuda(), freq.cuda(), norm="l2")
    o, _ = delta.gated_delta_rule(q, k, v, lg, lbe, None, seq.cuda(), nseqs=3)
    got = torch.autograd.grad(o, leaves, do.cuda())
    torch.cuda.synchronize()
    # the oracles, chained
    n64 = lambda t: t.double().numpy()  # noqa: E731
    xs, s = [n64(t) for t in (x, w, bias)], seq.numpy()
    yr = oc.forward(*xs, s, "silu")
    vr, kr, qr = yr[..., :64].reshape(1, L, H, P), yr[..., 64:128].reshape(1, L, G, N), yr[..., 128:].reshape(1, L, G, N)
    more = (pos.numpy(), n64(freq))
    qn, kn = on.forward(qr, n64(wq), *more, norm="l2"), on.forward(kr, n64(wk), *more, norm="l2")
    ref = od.forward(qn, kn, vr, n64(g), n64(beta), None, s)
    gr = od.backward(qn, kn, vr, n64(g), n64(beta), n64(do), None, s)
    dq, dwq = on.backward(qr, n64(wq), *more, gr["dq"], norm="l2")
    dk, dwk = on.backward(kr, n64(wk), *more, gr["dk"], norm="l2")
    dy = np.concatenate([t.reshape(1, L, -1) for t in (gr["dv"], dk, dq)], -1)
    gc = oc.backward(*xs, s, dy, "silu")
    # four operators, each within (N + 128) 2^-24 of its own result, forward and back
    tol = 8 * (N + 128) * 2.0 ** -24
    for name, a, r in zip(("o", "dx", "dw", "dbias", "dg", "dbeta", "dwq", "dwk"), (o, *got),
                          (ref["o"], gc["dx"], gc["dw"], gc["dbias"], gr["dg"], gr["dbeta"], dwq, dwk)):
        err = np.linalg.norm(f64(a) - r) / np.linalg.norm(r)
        print(f"  {name}: {err:.2e} (tolerance {tol:.1e})", flush=True)
        assert err <= tol, name
