"""NaN and infinite values in the gated linear recurrence: h_t = a_t h_{t-1} + m_t u_t is taken as it is written, so
one stays until its sequence ends (in the gradients: begins), however far that is, and however small the decays'
product has become on the way.  Which elements are finite is compared with the row-by-row oracle; an infinity may come
out as a NaN (zero times it), so of the others nothing more is asked."""
import numpy as np
import pytest
import torch

from oracle import recurrence as orc
from state_space_model_mamba_amd import recurrence as rec

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
BAD = {"nan": float("nan"), "inf": float("inf")}
KEYS = ("dx", "dg", "d_in_gate", "ddecay", "d_initial_states")


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(L, C, io, gate, lengths, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    t = IO[io]
    # decays around one half: the product of 64 rows is below 2^-40, that of 300 below float32's range
    g = -torch.nn.functional.softplus(rn(1, L, C)) if gate == "log" else rn(1, L, C).to(t)
    return {"x": rn(1, L, C).to(t), "g": g, "in_gate": rn(1, L, C).to(t), "decay": -1 - torch.rand((C,), generator=gen) if gate == "decay" else None,
            "h0": rn(len(lengths), C), "dfinal": rn(len(lengths), C), "dy": rn(1, L, C).to(t),
            "seq": torch.repeat_interleave(torch.arange(len(lengths), dtype=torch.int32), torch.tensor(lengths))[None].contiguous()}


def run(d, **kw):
    c = {k: None if v is None else v.cuda() for k, v in d.items()}
    r = rec.linrec_fwd(c["x"], c["g"], c["in_gate"], c["decay"], c["h0"], c["seq"], want_final_states=True, want_chunk_states=True, **kw)
    args = (c["x"], c["g"], c["in_gate"], c["decay"], c["dy"], c["h0"], c["seq"], c["dfinal"])
    g, again = rec.linrec_bwd(*args, r["chunk_states"], **kw), rec.linrec_bwd(*args, **kw)
    torch.cuda.synchronize()
    return {"y": r["y"], "final_states": r["final_states"], **g}, again


def same_pattern(d, label, **kw):
    print(f"[case] {label}", flush=True)
    got, again = run(d, **kw)
    h = {k: f64(v) for k, v in d.items()}
    seq = d["seq"].numpy()
    with np.errstate(all="ignore"):
        ref = orc.forward(h["x"], h["g"], h["in_gate"], h["decay"], h["h0"], seq, **kw)
        ref.update(orc.backward(h["x"], h["g"], h["in_gate"], h["decay"], h["dy"], h["h0"], seq, h["dfinal"], **kw))
    for k, t in got.items():
        if t is None:
            continue
        finite, want = np.isfinite(f64(t)), np.isfinite(ref[k])
        assert (finite == want).all(), f"{label} {k}: {int((finite != want).sum())} elements, the first at {np.argwhere(finite != want)[0]}"
        if k in again:
            assert (np.isfinite(f64(again[k])) == want).all(), f"{label} {k} without the kept states"


# lengths of one chunk, of the layout for up to 256 rows, and of several chunks in either direction
@pytest.mark.parametrize("lengths", [[60], [200], [700], [300, 5, 395]])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate,scale", [("sigmoid", "one"), ("decay", "unit"), ("log", "complement")])
def test_a_bad_value_lasts_to_its_sequences_end(gate, scale, io, lengths):
    L, C = sum(lengths), 16
    for name in ("x", "dy", "g"):
        for kind, bad in BAD.items():
            if name == "g" and kind == "inf":   # gates of infinity are closed or open ones
                continue
            for row in (10, L - 11):
                d = make(L, C, io, gate, lengths, seed=L)
                d[name][0, row, 5] = bad
                same_pattern(d, f"{gate} {scale} {io} {lengths}: {kind} in {name} at row {row}", gate=gate, input_scale=scale)


@pytest.mark.parametrize("name", ["h0", "dfinal"])
def test_a_bad_state_lasts_to_its_sequences_end(name):
    for kind, bad in BAD.items():
        d = make(900, 16, "f32", "sigmoid", [500, 400], seed=1)
        d[name][1, 3] = bad
        same_pattern(d, f"{kind} in {name}", gate="sigmoid", input_scale="one")


@pytest.mark.parametrize("L", [100, 200, 600])
def test_a_decay_of_zero_drops_what_is_finite_only(L):
    # exp(-inf) = 0: zero times a finite state is nothing of it, zero times an infinity is a NaN; the large decays around it
    # make each product of a chunk zero as well
    for kind, bad in BAD.items():
        for row, drop in ((10, 40), (40, 10)):
            d = make(L, 16, "f32", "log", [L], seed=2)
            d["g"][0, drop] = float("-inf")
            d["g"][0, drop + 2::3] = -200.0
            d["x"][0, row, 5] = bad
            same_pattern(d, f"{kind} at row {row}, a decay of zero at {drop}, {L} rows", gate="log", input_scale="one")


def test_in_one_call_or_in_many():
    # the same rows whole, in two calls and by tokens: the same elements are finite
    L, C, kw = 640, 16, dict(gate="sigmoid", input_scale="complement")
    d = {k: v.cuda() if v is not None else None for k, v in make(L, C, "f32", "sigmoid", [L], seed=3).items()}
    d["x"][0, 10, 5], d["x"][0, 300, 7] = float("nan"), float("inf")
    part = lambda lo, hi, h: rec.linrec_fwd(d["x"][:, lo:hi], d["g"][:, lo:hi], initial_states=h, want_final_states=True, **kw)  # noqa: E731
    whole, one = part(0, L, d["h0"]), part(0, 200, d["h0"])
    two = part(200, L, one["final_states"])
    pool, ys = d["h0"].clone(), []
    for t in range(0, L, 64):
        ys.append(rec.linrec_step(d["x"][:, t:t + 64], d["g"][:, t:t + 64], pool, **kw))
    finite = lambda t: torch.isfinite(t)  # noqa: E731
    ref = finite(torch.cat(ys, 1))
    assert not ref[0, 10:, 5].any() and not ref[0, 300:, 7].any() and int((~ref).sum()) == L - 10 + L - 300
    assert torch.equal(finite(whole["y"]), ref) and torch.equal(finite(torch.cat([one["y"], two["y"]], 1)), ref)
    assert torch.equal(finite(whole["final_states"]), finite(pool)) and torch.equal(finite(two["final_states"]), finite(pool))
