"""The norms, the convolution and the gated linear recurrence as a recurrent block
uses them together: training against float64 on the CPU (outputs and all
gradients), and a prompt followed by single tokens against the whole sequence.

Tolerances, on the 2-norm of the difference over that of the result: no output
or gradient here is formed by more than 64 float32 roundings for each of the rows
that reach it (sums over 64 channels included), so rows * 64 * 2^-24; with bf16
each of the five tensors between the operators adds its rounding, 2^-8.
"""
import pytest
import torch
import torch.nn.functional as F

from state_space_model_mamba_amd import block_norm, conv1d, recurrence

pytestmark = pytest.mark.gpu
D, C, ALPHA, EPS = 64, 128, 0.5, 1e-5


def parameters(seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    return {"norm": 1 + 0.1 * rn(D), "into": rn(D, 4 * C) / 8, "filter": rn(C, 4) / 2, "shift": rn(C) / 4, "decay": -8 * torch.rand((C,), generator=gen),
            "gate_norm": 1 + 0.1 * rn(C), "out": rn(C, D) / 11, "post": 1 + 0.1 * rn(D)}


def block(x, residual, w, seq_idx=None, h0=None, nseqs=None):
    y, r = block_norm.add_norm(x, residual, w["norm"], eps=EPS)
    p = y @ w["into"].to(y.dtype)
    u, z, g, i = p.split(C, dim=-1)
    u = conv1d.causal_conv1d(u.contiguous(), w["filter"], w["shift"], seq_idx)
    h, final = recurrence.linear_recurrence(u, g, i, w["decay"], h0, seq_idx, gate="decay", input_scale="unit", nseqs=nseqs)
    n = block_norm.gated_norm(h, z, w["gate_norm"], groups=4, eps=EPS)
    return block_norm.gated_norm(n @ w["out"].to(n.dtype), None, w["post"], residual=r, scale=ALPHA, eps=EPS, norm="layer"), final


def rms(u, groups=1):
    v = u.unflatten(-1, (groups, -1))
    return (v / (v.square().mean(-1, keepdim=True) + EPS).sqrt()).flatten(-2)


def block64(x, residual, w, lengths, h0):
    """The same in float64, sequence by sequence and row by row."""
    r = x + residual
    u, z, g, i = ((rms(r) * w["norm"]) @ w["into"]).split(C, dim=-1)
    hs, finals, at = [], [], 0
    for s, n in enumerate(lengths):
        part = slice(at, at + n)
        v = F.pad(u[0, part].T, (3, 0))
        v = F.silu(F.conv1d(v[None], w["filter"][:, None], w["shift"], groups=C))[0].T
        la = w["decay"] * torch.sigmoid(g[0, part])
        b = (-torch.expm1(2 * la)).sqrt() * v * torch.sigmoid(i[0, part])
        h = h0[s]
        for t in range(n):
            h = la[t].exp() * h + b[t]
            hs.append(h)
        finals.append(h)
        at += n
    n = rms(torch.stack(hs)[None] * F.silu(z), 4) * w["gate_norm"]
    o = n @ w["out"]
    return r + ALPHA * F.layer_norm(o, (D,), w["post"], None, EPS), torch.stack(finals)


def close(a, b, tol, label):
    err = float((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm())
    print(f"  {label}: {err:.2e} (tolerance {tol:.1e})", flush=True)
    assert err <= tol, label


def test_a_training_step_of_packed_sequences():
    lengths = [70, 1, 129]
    L = sum(lengths)
    gen = torch.Generator().manual_seed(1)
    x, res, dout = (torch.randn((1, L, D), generator=gen) for _ in range(3))
    h0, dfinal = torch.randn((3, C), generator=gen), torch.randn((3, C), generator=gen)
    seq = torch.repeat_interleave(torch.arange(3, dtype=torch.int32), torch.tensor(lengths))[None].contiguous()
    w = parameters()
    ref_leaves = [t.double().requires_grad_(True) for t in (x, res, h0, *w.values())]
    ref = block64(ref_leaves[0], ref_leaves[1], dict(zip(w, ref_leaves[3:])), lengths, ref_leaves[2])
    ref_grads = torch.autograd.grad(ref, ref_leaves, (dout.double(), dfinal.double()))
    leaves = [t.cuda().requires_grad_(True) for t in (x, res, h0, *w.values())]
    out = block(leaves[0], leaves[1], dict(zip(w, leaves[3:])), seq.cuda(), leaves[2])
    grads = torch.autograd.grad(out, leaves, (dout.cuda(), dfinal.cuda()))
    torch.cuda.synchronize()
    tol = L * 64 * 2.0 ** -24
    for a, b, name in zip((*out, *grads), (*ref, *ref_grads), ("out", "final", "dx", "dresidual", "dh0", *("d" + k for k in w))):
        close(a, b, tol, name)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_prompt_and_single_tokens(dtype):
    b, L, tokens = 3, 90, 5
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((b, L + tokens, D), generator=gen).to(dtype).cuda()
    w = {k: v.cuda() for k, v in parameters().items()}

    def parts(x):
        y, r = block_norm.add_norm_fwd(x, None, w["norm"], eps=EPS, residual_dtype=torch.float32)
        return r, (y @ w["into"].to(dtype)).split(C, dim=-1)

    def rest(h, z, r):
        n = block_norm.gated_norm_fwd(h, z, w["gate_norm"], groups=4, eps=EPS)
        return block_norm.gated_norm_fwd(n @ w["out"].to(dtype), None, w["post"], None, r, ALPHA, eps=EPS)

    kw = dict(gate="decay", input_scale="unit")
    r, (u, z, g, i) = parts(x)
    whole = rest(recurrence.linrec_fwd(u, g, i, w["decay"], **kw)["y"], z, r)
    r, (u, z, g, i) = parts(x[:, :L])
    first = recurrence.linrec_fwd(u, g, i, w["decay"], want_final_states=True, **kw)
    outs, pool = [rest(first["y"], z, r)], torch.zeros((7, C), device="cuda")
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    pool[slots.long()] = first["final_states"]
    for t in range(L, L + tokens):
        r, (u, z, g, i) = parts(x[:, t:t + 1])
        outs.append(rest(recurrence.linrec_step(u, g, pool, i, w["decay"], slots, **kw), z, r))
    close(torch.cat(outs, 1), whole.double().cpu(), (L + tokens) * 64 * 2.0 ** -24 + (5 * 2.0 ** -8 if dtype == torch.bfloat16 else 0), str(dtype))
