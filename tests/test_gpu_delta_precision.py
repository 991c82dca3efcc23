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
from tests.test_gpu_delta import args, cuda, f64, make

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
