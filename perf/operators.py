"""The cases on which the gated delta rule and the per-head norm with rotation are measured.

Three operators, next to the SSD scan and the causal convolution of this package:

* the gated delta rule over whole sequences ("prefill": forward with the final states; "train":
  forward and all gradients).  Per sequence and head, S in R^{N x P}, S_0 the initial state:
      Sd_t = exp(g_t) S_{t-1},  e_t = v_t - Sd_t^T k_t,  S_t = Sd_t + beta_t k_t e_t^T,
      o_t = scale S_t^T q_t
* its form for few tokens on a pool of states kept in memory ("step": one token a sequence, or a few
  drafted ones)
* the norm of every query and key head with the position rotation in the same pass ("norm": forward;
  "norm_train": forward and all gradients)

`own` is False: run() computes the plain forms, in elementary torch operations.  `own` is True: run()
calls the package's entry points.
"""
import math

import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def delta_case(name, kind, dtype, batch, seqlen, heads, headdim, groups, dstate, nseqs=0, initial=False, packed=False):
    return {"name": name, "kind": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen, "heads": heads, "headdim": headdim,
            "groups": groups, "dstate": dstate, "nseqs": nseqs, "initial": initial, "packed": packed}


def step_case(name, dtype, batch, tokens, heads, headdim, groups, dstate, slots, holes=False):
    return {"name": name, "kind": "step", "dtype": dtype, "batch": batch, "tokens": tokens, "heads": heads, "headdim": headdim,
            "groups": groups, "dstate": dstate, "slots": slots, "holes": holes}


def norm_case(name, kind, dtype, batch, seqlen, qheads, kheads, dstate, rot, norm, interleaved, far):
    return {"name": name, "kind": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen, "qheads": qheads, "kheads": kheads,
            "dstate": dstate, "rot": rot, "norm": norm, "interleaved": interleaved, "far": far}


def listed():
    return [
        # a short odd prompt on a small layer: latency counts
        delta_case("prefill_L200_H4", "prefill", "bf16", 1, 200, 4, 64, 2, 128),
        # a prompt on the layer of the bf16_L2048_H128 workload; q, k and v are slices of the convolution's output
        delta_case("prefill_L2048_H128", "prefill", "bf16", 1, 2048, 128, 64, 8, 128, packed=True),
        # seven prompts of uneven lengths packed in one row, each resumed from a state (64 heads that share one q and k)
        delta_case("prefill_varlen7_L16384", "prefill", "bf16", 1, 16384, 64, 64, 1, 128, nseqs=7, initial=True),
        # training, the tiny_f32_L256 workload's layer in fp32
        delta_case("train_f32_L256", "train", "f32", 1, 256, 4, 16, 1, 16),
        # training on packed documents, wide values, a head of its own for every key; odd total length
        delta_case("train_varlen5_L1999_P128", "train", "bf16", 1, 1999, 16, 128, 16, 128, nseqs=5, initial=True),
        # training, the bf16_B2_L4096_H128 workload's layer
        delta_case("train_B2_L4096_H128", "train", "bf16", 2, 4096, 128, 64, 8, 128),
        # training, the bf16_L16384_H128 workload's layer: the largest
        delta_case("train_L16384_H128", "train", "bf16", 1, 16384, 128, 64, 8, 128),
        # one token of one sequence: the smallest serving call
        step_case("step_B1_H128", "bf16", 1, 1, 128, 64, 8, 128, 16),
        # one token of a padded batch of 64 sequences, a few rows of it empty
        step_case("step_B64_H128", "bf16", 64, 1, 128, 64, 8, 128, 80, holes=True),
        # four drafted tokens each of 24 sequences
        step_case("step_B24_T4_H64", "bf16", 24, 4, 64, 64, 1, 128, 32),
        # the q and k heads of one decoded token for each of 16 sequences, far into their contexts
        norm_case("norm_B16_T1", "norm", "bf16", 16, 1, 8, 8, 128, 64, "rms", False, 1000003),
        # training, the q and k heads of the 16384-token layer, in full rotation
        norm_case("norm_train_L16384", "norm_train", "bf16", 1, 16384, 8, 8, 128, 128, "rms", False, 0),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "train", "train", "step", "step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dstate = rng.choice([16, 40, 64, 96, 128, 128])
    if kind in ("norm", "norm_train"):
        batch = rng.choice([1, 1, 2, 3])
        rot = rng.choice([0, 16, dstate // 2 // 2 * 2, dstate])
        return {k: v for k, v in norm_case("", kind, dtype, batch, log_int(rng, 1, 16384 // batch), rng.choice([1, 3, 4, 8, 16]), rng.choice([1, 2, 4, 8]),
                                           dstate, min(rot, dstate), rng.choice(["rms", "l2"]), rng.random() < 0.5, rng.choice([0, 777, 1000003])).items() if k != "name"}
    groups = rng.choice([1, 2, 4, 8])
    heads = groups * rng.choice([1, 2, 3, 8])
    headdim = rng.choice([16, 24, 64, 64, 128])
    if kind == "step":
        batch = log_int(rng, 1, 64)
        case = step_case("", dtype, batch, rng.choice([1, 1, 1, 2, 5]), heads, headdim, groups, dstate, batch + rng.randint(1, 16), rng.random() < 0.5)
    else:
        batch, nseqs = rng.choice([1, 1, 2, 3]), 0
        if rng.random() < 0.4:
            batch, nseqs = 1, rng.randint(2, 9)
        seqlen = log_int(rng, 1 if not nseqs else 40, 8192 // batch)
        case = delta_case("", kind, dtype, batch, seqlen, heads, headdim, groups, dstate, nseqs, rng.random() < 0.5, rng.random() < 0.3)
    return {k: v for k, v in case.items() if k != "name"}


def work(c):
    size = 2 if c["dtype"] == "bf16" else 4
    n = c["dstate"]
    if c["kind"] in ("norm", "norm_train"):
        tokens = c["batch"] * c["seqlen"]
        values = tokens * (c["qheads"] + c["kheads"]) * n
        train = c["kind"] == "norm_train"
        # read x and write y; for gradients also read dy and write dx; the positions once
        return {"bytes": values * size * (4 if train else 2) + 4 * tokens, "flops": values * (24 if train else 8)}
    h, p, g = c["heads"], c["headdim"], c["groups"]
    if c["kind"] == "step":
        live = c["batch"] - (c["batch"] // 9 if c["holes"] else 0)
        tokens = live * c["tokens"]
        return {"bytes": 2 * 4 * live * h * p * n + tokens * ((2 * g * n + 2 * h * p) * size + 8 * h), "flops": tokens * h * p * n * 7}
    tokens, seqs = c["batch"] * c["seqlen"], c["nseqs"] or c["batch"]
    qk, v, gates, states = tokens * 2 * g * n * size, tokens * h * p * size, tokens * 2 * h * 4, seqs * h * p * n * 4
    if c["kind"] == "prefill":
        return {"bytes": qk + 2 * v + gates + states * (2 if c["initial"] else 1), "flops": tokens * h * p * n * 7}
    # gradients: q, k, v, g, beta and do read, o, dq, dk, dv, dg and dbeta written, and the states both ways
    return {"bytes": 2 * qk + 4 * v + 2 * gates + states * (2 if c["initial"] else 0), "flops": tokens * h * p * n * 25}


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def gates(shape, gen):
    """g and beta as a layer's front-end makes them: the log decay A softplus(z + bias), and a sigmoid."""
    h = shape[-1]
    z = torch.randn(shape, generator=gen, device="cuda") * 0.5
    u = torch.rand((h,), generator=gen, device="cuda", dtype=torch.float64) * (1e-1 - 1e-3) + 1e-3
    a = torch.exp(torch.rand((h,), generator=gen, device="cuda") * math.log(16.0))
    dt = torch.nn.functional.softplus(z + torch.log(torch.expm1(u)).float())
    return (-a * dt).contiguous(), torch.sigmoid(torch.randn(shape, generator=gen, device="cuda")).contiguous()


def unit_rows(shape, gen):
    x = torch.randn(shape, generator=gen, device="cuda")
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def lengths_of(c, seed):
    """The packed sequences' lengths: uneven, one token at least, the case's tokens in all."""
    n, gen = c["nseqs"], torch.Generator().manual_seed(int(seed) + 1)
    cuts = torch.randperm(c["seqlen"] - 1, generator=gen)[: n - 1].sort().values.tolist()
    edges = [0] + [x + 1 for x in cuts] + [c["seqlen"]]
    return [edges[i + 1] - edges[i] for i in range(n)]


def prepare(c, seed):
    gen, io, n = generator(seed), IO[c["dtype"]], c["dstate"]
    if c["kind"] in ("norm", "norm_train"):
        b, L, rot = c["batch"], c["seqlen"], c["rot"]
        s = {"case": c, "q": torch.randn((b, L, c["qheads"], n), generator=gen, device="cuda").to(io),
             "k": torch.randn((b, L, c["kheads"], n), generator=gen, device="cuda").to(io),
             "q_weight": None, "k_weight": None, "inv_freq": None, "positions": None}
        if c["norm"] == "rms":
            s["q_weight"] = 1 + 0.1 * torch.randn((n,), generator=gen, device="cuda")
            s["k_weight"] = 1 + 0.1 * torch.randn((n,), generator=gen, device="cuda")
        if rot:
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
            s["positions"] = (torch.arange(L, dtype=torch.int32, device="cuda")[None, :] +
                              torch.randint(0, c["far"] + 1, (b, 1), generator=gen, device="cuda", dtype=torch.int32)).contiguous()
        if c["kind"] == "norm_train":
            s["dq"] = torch.randn(s["q"].shape, generator=gen, device="cuda").to(io)
            s["dk"] = torch.randn(s["k"].shape, generator=gen, device="cuda").to(io)
            s["leaves"] = [t.requires_grad_(True) for t in (s["q"], s["k"], s["q_weight"], s["k_weight"]) if t is not None]
        return s
    h, p, g = c["heads"], c["headdim"], c["groups"]
    b, L = c["batch"], c["tokens"] if c["kind"] == "step" else c["seqlen"]
    q, k = unit_rows((b, L, g, n), gen).to(io), unit_rows((b, L, g, n), gen).to(io)
    v = torch.randn((b, L, h, p), generator=gen, device="cuda").to(io)
    gate, beta = gates((b, L, h), gen)
    s = {"case": c, "q": q, "k": k, "v": v, "g": gate, "beta": beta}
    if c["kind"] == "step":
        s["states"] = torch.randn((c["slots"], h, p, n), generator=gen, device="cuda") * 0.1
        index = torch.randperm(c["slots"], generator=gen, device="cuda")[:b].to(torch.int32)
        if c["holes"]:
            index[torch.randperm(b, generator=gen, device="cuda")[: b // 9]] = -1
        s["state_indices"] = index.contiguous()
        return s
    if c["packed"]:  # slices of one row of channels, as they leave the convolution
        row = torch.cat([v.reshape(b, L, h * p), k.reshape(b, L, g * n), q.reshape(b, L, g * n)], dim=-1).contiguous()
        s["v"] = row[..., : h * p].unflatten(-1, (h, p))
        s["k"] = row[..., h * p: h * p + g * n].unflatten(-1, (g, n))
        s["q"] = row[..., h * p + g * n:].unflatten(-1, (g, n))
    s["nseqs"] = c["nseqs"] or b
    s["lengths"] = lengths_of(c, seed) if c["nseqs"] else None
    s["seq_idx"] = None
    if c["nseqs"]:
        s["seq_idx"] = torch.repeat_interleave(torch.arange(c["nseqs"], dtype=torch.int32), torch.tensor(s["lengths"])).reshape(1, L).cuda()
    s["initial_states"] = torch.randn((s["nseqs"], h, p, n), generator=gen, device="cuda") * 0.1 if c["initial"] else None
    if c["kind"] == "train":
        s["do"] = torch.randn((b, L, h, p), generator=gen, device="cuda").to(io)
        s["leaves"] = [t.requires_grad_(True) for t in ([s["q"].detach(), s["k"].detach(), s["v"].detach(), gate, beta] +
                                                       ([s["initial_states"]] if c["initial"] else []))]
        s["q"], s["k"], s["v"] = s["leaves"][:3]
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
CHUNK = 64


def chunked(x, pad):
    """(S, T, H, ...) -> (S, H, chunks, CHUNK, ...) in 32 bits, rows past T zero."""
    x = torch.cat([x, x.new_zeros((x.shape[0], pad) + tuple(x.shape[2:]))], dim=1) if pad else x
    return x.unflatten(1, (-1, CHUNK)).movedim(3, 1).float()


def plain_delta(q, k, v, g, beta, s0):
    """The gated delta rule of S sequences of T tokens each, all of (S, T, ...): o and the last states in 32 bits.

    Within a chunk of tokens, with c_i the sum of g up to i and G_ij = exp(c_i - c_j), the corrections
    u_i = beta_i e_i solve (I + A) u = beta (v - exp(c) k S), A_ij = beta_i G_ij k_i.k_j for j < i, and the
    inverse of I + A is the product of (I - A), (I + A^2), (I + A^4) .. (I + A^32): A^64 is zero."""
    heads, groups, n, T = v.shape[2], q.shape[2], q.shape[3], q.shape[1]
    q, k = (t.float().repeat_interleave(heads // groups, dim=2) for t in (q, k))
    pad = -T % CHUNK
    q, k, v, g, beta = (chunked(t, pad) for t in (q, k, v, g, beta))
    c = g.double().cumsum(-1)
    low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=q.device).tril()
    decay = torch.where(low, (c[..., :, None] - c[..., None, :]).masked_fill(~low, 0).exp(), 0.0).float()
    kt = k.transpose(-1, -2).contiguous()
    A = (beta[..., None] * decay * (k @ kt)).tril(-1)
    A2 = A @ A
    A4 = A2 @ A2
    A8 = A4 @ A4
    A16 = A8 @ A8
    A32 = A16 @ A16
    X = A2 - A @ A2 - A  # (I - A)(I + A^2) - I
    X = A4 + X @ A4 + X
    X = A8 + X @ A8 + X
    X = A16 + X @ A16 + X
    X = A32 + X @ A32 + X
    attn = decay * (q @ kt)
    into = c.exp().float()[..., None]  # what is left of the entering state at each row
    kin, qin = beta[..., None] * into * k, into * q
    kin, vb = kin + X @ kin, beta[..., None] * v
    vb = vb + X @ vb
    kout = ((c[..., -1:] - c).exp().float()[..., None] * k).transpose(-1, -2).contiguous()
    last = c[..., -1].exp().float()[..., None, None]
    state, out = s0.transpose(-1, -2), []
    for i in range(q.shape[2]):  # a chunk's entering state is the last one's result: in order
        u = vb[:, :, i] - kin[:, :, i] @ state
        out.append(qin[:, :, i] @ state + attn[:, :, i] @ u)
        state = last[:, :, i] * state + kout[:, :, i] @ u
    o = torch.stack(out, dim=2).movedim(1, 3).flatten(1, 2)[:, :T] / math.sqrt(n)
    return o, state.transpose(-1, -2).contiguous()


def rows_of(lengths, device):
    """For packed sequences of one row: (S, longest) indices into its tokens, the row past the last for none; and where each token went."""
    at, longest = [], max(lengths)
    edges = torch.tensor([0] + lengths, device=device).cumsum(0)
    step = torch.arange(longest, device=device)
    inside = step[None, :] < (edges[1:] - edges[:-1])[:, None]
    return torch.where(inside, edges[:-1, None] + step[None, :], edges[-1]), inside


def plain_sequences(s):
    q, k, v, g, beta = (s[x] for x in ("q", "k", "v", "g", "beta"))
    s0 = s["initial_states"]
    if s0 is None:
        s0 = torch.zeros((s["nseqs"], v.shape[2], v.shape[3], q.shape[3]), device=q.device)
    if s["lengths"] is None:
        o, last = plain_delta(q, k, v, g, beta, s0)
    else:
        # every sequence in a row of its own; a row of zeros (no decay, no key) leaves the state as it is
        index, inside = rows_of(s["lengths"], q.device)
        apart = lambda t: torch.cat([t[0].float(), t.new_zeros((1,) + tuple(t.shape[2:])).float()])[index]  # noqa: E731
        o, last = plain_delta(apart(q), apart(k), apart(v), apart(g), apart(beta), s0)
        o = o[inside][None]
    return o.to(v.dtype), last


def plain_step(s):
    q, k, v, g, beta, states, index = (s[x] for x in ("q", "k", "v", "g", "beta", "states", "state_indices"))
    rep, n = v.shape[2] // q.shape[2], q.shape[3]
    live = index >= 0
    at = index.clamp(min=0).long()
    qf, kf = q.float().repeat_interleave(rep, dim=2), k.float().repeat_interleave(rep, dim=2)
    S, out = states[at], []
    for t in range(q.shape[1]):  # a token's state is the one before's result: in order
        Sd = S * g[:, t].exp()[..., None, None]
        e = v[:, t].float() - (Sd * kf[:, t, :, None, :]).sum(-1)
        S = Sd + (beta[:, t, :, None] * e)[..., None] * kf[:, t, :, None, :]
        out.append((S * qf[:, t, :, None, :]).sum(-1) / math.sqrt(n))
    o = torch.where(live[:, None, None, None], torch.stack(out, dim=1), 0.0).to(v.dtype)
    states[at[live]] = S[live]
    return o, states


def plain_norm(x, weight, norm, positions, inv_freq, interleaved, eps):
    f = x.float()
    square = (f * f).mean(-1, keepdim=True) if norm == "rms" else (f * f).sum(-1, keepdim=True)
    f = f * torch.rsqrt(square + eps)
    if weight is not None:
        f = f * weight
    if inv_freq is not None:
        angle = positions.double()[..., None, None] * inv_freq.double()
        c, s, rot = angle.cos().float(), angle.sin().float(), 2 * inv_freq.numel()
        r, rest = f[..., :rot], f[..., rot:]
        a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])
        a, b = a * c - b * s, b * c + a * s
        r = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
        f = torch.cat([r, rest], dim=-1)
    return f.to(x.dtype)


EPS = 1e-6


def run(s):
    c = s["case"]
    kind = c["kind"]
    if own:
        from state_space_model_mamba_amd import delta, qk_norm
        if kind == "prefill":
            r = delta.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["initial_states"], s["seq_idx"], nseqs=s["nseqs"], want_final_states=True)
            return {"o": r["o"], "final_states": r["final_states"]}
        if kind == "train":
            o, _ = delta.gated_delta_rule(*s["leaves"][:5], s["initial_states"], s["seq_idx"], nseqs=s["nseqs"])
            return {"o": o, "grads": torch.autograd.grad(o, s["leaves"], s["do"])}
        if kind == "step":
            return {"o": delta.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"], s["state_indices"]), "states": s["states"]}
        more = dict(norm=c["norm"], eps=EPS, interleaved=c["interleaved"])
        if kind == "norm":
            y = qk_norm.qk_norm_rope_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"], **more)
            return {"q": y[0], "k": y[1]}
        y = qk_norm.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"], **more)
        return {"q": y[0], "k": y[1], "grads": torch.autograd.grad(y, s["leaves"], (s["dq"], s["dk"]))}
    if kind == "prefill":
        o, last = plain_sequences(s)
        return {"o": o, "final_states": last}
    if kind == "train":
        o, _ = plain_sequences(s)
        return {"o": o, "grads": torch.autograd.grad(o, s["leaves"], s["do"])}
    if kind == "step":
        o, states = plain_step(s)
        return {"o": o, "states": states}
    q = plain_norm(s["q"], s["q_weight"], c["norm"], s["positions"], s["inv_freq"], c["interleaved"], EPS)
    k = plain_norm(s["k"], s["k_weight"], c["norm"], s["positions"], s["inv_freq"], c["interleaved"], EPS)
    if kind == "norm":
        return {"q": q, "k": k}
    return {"q": q, "k": k, "grads": torch.autograd.grad((q, k), s["leaves"], (s["dq"], s["dk"]))}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def recur(q, k, v, g, beta, S, do=None):
    """The recurrence of the top of this file for (B, T, ...) in 64 bits, token by token; with do the adjoint recurrence too.

    With D the gradient of S_t (what later tokens gave, plus q_t do_t^T scale), reading the recurrence backwards:
    du = D^T k, de = beta du, D' = D - k de^T is that of Sd_t, dg = <D', Sd_t>, and exp(g) D' goes on to S_{t-1}."""
    q, k, v, g, beta, S = (t.detach().double() for t in (q, k, v, g, beta, S))
    rep, scale, T, G = v.shape[2] // q.shape[2], 1.0 / math.sqrt(q.shape[3]), q.shape[1], q.shape[2]
    q, k = q.repeat_interleave(rep, dim=2), k.repeat_interleave(rep, dim=2)
    o = torch.zeros_like(v)
    span, kept = 256, []

    def token(S, t):
        Sd = S * g[:, t, :, None, None].exp()
        e = v[:, t] - torch.einsum("bhpn,bhn->bhp", Sd, k[:, t])
        return Sd, e, Sd + (beta[:, t, :, None] * e)[..., None] * k[:, t, :, None, :]

    for t in range(T):
        if do is not None and t % span == 0:
            kept.append(S)
        _, _, S = token(S, t)
        o[:, t] = scale * torch.einsum("bhpn,bhn->bhp", S, q[:, t])
    if do is None:
        return o, S
    do, D = do.detach().double(), torch.zeros_like(S)
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    for first in range((T - 1) // span * span, -1, -span):
        S, saved = kept[first // span], []
        for t in range(first, min(T, first + span)):
            Sd, e, S = token(S, t)
            saved.append((Sd, e, S))
        for t in range(min(T, first + span) - 1, first - 1, -1):
            Sd, e, S = saved.pop()
            D = D + scale * do[:, t, :, :, None] * q[:, t, :, None, :]
            dq[:, t] = scale * torch.einsum("bhpn,bhp->bhn", S, do[:, t])
            du = torch.einsum("bhpn,bhn->bhp", D, k[:, t])
            db[:, t] = (du * e).sum(-1)
            de = beta[:, t, :, None] * du
            dv[:, t] = de
            dk[:, t] = torch.einsum("bhpn,bhp->bhn", D, beta[:, t, :, None] * e) - torch.einsum("bhpn,bhp->bhn", Sd, de)
            D = D - de[..., None] * k[:, t, :, None, :]
            dg[:, t] = (D * Sd).sum((-1, -2))
            D = D * g[:, t, :, None, None].exp()
    sums = lambda x: x.unflatten(2, (G, rep)).sum(3)  # noqa: E731
    return o, [sums(dq), sums(dk), dv, dg, db, D]


def exact_norm(x, weight, norm, eps, positions, inv_freq, interleaved, dy=None):
    """Norm and rotation in 64 bits as complex products; with dy the gradients of x and weight."""
    x = x.detach().double()
    n = x.shape[-1]
    m = n if norm == "rms" else 1
    r = ((x.pow(2).sum(-1, keepdim=True)) / m + eps).pow(-0.5)
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.detach().double()

    def turn(z, sign):
        if inv_freq is None:
            return z
        rot = 2 * inv_freq.numel()
        phase = torch.polar(torch.ones((), dtype=torch.float64, device=z.device), sign * positions.double()[:, :, None, None] * inv_freq.double())
        if interleaved:
            pairs = z[..., :rot].unflatten(-1, (rot // 2, 2))
        else:
            pairs = z[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
        turned = turned.flatten(-2) if interleaved else turned.transpose(-1, -2).flatten(-2)
        return torch.cat([turned, z[..., rot:]], dim=-1)

    y = turn(x * r * w, 1)
    if dy is None:
        return y
    dz = turn(dy.double(), -1)
    dx = r * w * dz - x * r.pow(3) / m * (w * dz * x).sum(-1, keepdim=True)
    return y, dx, (dz * x * r).sum((0, 1, 2))


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] in ("norm", "norm_train"):
        train = c["kind"] == "norm_train"
        q, k = (exact_norm(s[x], s[x + "_weight"], c["norm"], EPS, s["positions"], s["inv_freq"], c["interleaved"], s["d" + x] if train else None) for x in "qk")
        if not train:
            return {"q": q, "k": k}
        grads = [q[1], k[1]] + ([q[2], k[2]] if s["q_weight"] is not None else [])
        return {"q": q[0], "k": k[0], "grads": grads}
    if c["kind"] == "step":
        live = s["state_indices"] >= 0
        at = s["state_indices"][live].long()
        o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
        states = s["states"].double()
        o[live], states[at] = recur(*(s[x][live] for x in ("q", "k", "v", "g", "beta")), s["states"][at])
        return {"o": o, "states": states}
    inputs = [s[x] for x in ("q", "k", "v", "g", "beta")]
    h, p, n = c["heads"], c["headdim"], c["dstate"]
    s0 = s["initial_states"] if c["initial"] else torch.zeros((s["nseqs"], h, p, n), device="cuda")
    train = c["kind"] == "train"
    # sequence by sequence where they are packed, all rows at once where they are not
    parts, first = [], 0
    for i, length in enumerate(s["lengths"] or [c["seqlen"]]):
        part = slice(first, first + length)
        parts.append(recur(*(x[:, part] for x in inputs), s0[i: i + 1] if s["lengths"] else s0, s["do"][:, part] if train else None))
        first += length
    o = torch.cat([x[0] for x in parts], dim=1)
    if not train:
        return {"o": o, "final_states": torch.cat([x[1] for x in parts], dim=0)}
    grads = [torch.cat([x[1][j] for x in parts], dim=1) for j in range(5)]
    return {"o": o, "grads": grads + ([torch.cat([x[1][5] for x in parts], dim=0)] if c["initial"] else [])}
