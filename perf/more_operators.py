"""The cases on which the norms around a block and the gated linear recurrence are measured.

Next to the SSD scan, the causal convolution and the gated delta rule of this package:

* the norm before a block with the residual's sum in the same pass ("add_norm": forward, "add_norm_train": forward
  and all gradients):  r' = residual + s x,  y = norm(r') w + b
* the norm after a block with its gate, and with the residual's sum where the block ends there ("gated_norm",
  "gated_norm_train"), over groups of channels:
      n = norm(x act(z)) w + b   or   (norm(x) w + b) act(z),   out = s n   or   residual + s n
* the gated linear recurrence per channel ("recur": forward with the final states, "recur_train": forward and all
  gradients, "recur_step": few tokens on a pool of states), h_0 a sequence's initial state:
      h_t = a_t h_{t-1} + m_t u_t,   u = x  or  x sigmoid(i),   m = 1, 1 - a  or  sqrt(1 - a^2),
      a = exp(g), sigmoid(g)  or  exp(decay_c sigmoid(g))

`own` is False: run() computes the plain forms, in elementary torch operations.  `own` is True: run()
calls the package's entry points.
"""
import math

import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
ALPHA = 0.7   # the residual scale where it is one number


def norm_case(name, kind, dtype, batch, seqlen, width, groups=1, norm="rms", residual="none", scale="none", bias=False,
              gate="none", norm_first=False):
    return {"name": name, "kind": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen, "width": width, "groups": groups,
            "norm": norm, "residual": residual, "scale": scale, "bias": bias, "gate": gate, "norm_first": norm_first}


def recur_case(name, kind, dtype, batch, seqlen, channels, gate, input_scale, in_gate, nseqs=0, initial=False, packed=False):
    return {"name": name, "kind": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen, "channels": channels, "gate": gate,
            "input_scale": input_scale, "in_gate": in_gate, "nseqs": nseqs, "initial": initial, "packed": packed}


def step_case(name, dtype, batch, tokens, channels, gate, input_scale, in_gate, slots, holes=False):
    return {"name": name, "kind": "recur_step", "dtype": dtype, "batch": batch, "seqlen": tokens, "channels": channels, "gate": gate,
            "input_scale": input_scale, "in_gate": in_gate, "slots": slots, "holes": holes}


LARGEST = recur_case("recur_train_L16384_C8192", "recur_train", "bf16", 1, 16384, 8192, "decay", "unit", True)


def listed():
    return [
        # the norm before the next block for one decoded token, the residual stream in fp32: latency counts
        norm_case("add_norm_B1_D4096", "add_norm", "bf16", 1, 1, 4096, residual="f32"),
        # a batch of short prompts through an odd width, layer norm with its bias, one number as residual scale
        norm_case("add_norm_B6_L333_D1000", "add_norm", "f32", 6, 333, 1000, norm="layer", residual="io", scale="float", bias=True),
        # training at the 16384-token layer's width (its 8192 channels are twice the model's), a learned scale on each channel
        norm_case("add_norm_train_L16384_D4096", "add_norm_train", "bf16", 1, 16384, 4096, residual="f32", scale="vector"),
        # the gated norm of 64 decoded tokens behind the scan of 128 heads of 64, its 8 groups normed apart
        norm_case("gated_norm_B64_D8192_G8", "gated_norm", "bf16", 64, 1, 8192, groups=8, gate="silu"),
        # the same layer in training, the 16384-token workload
        norm_case("gated_norm_train_L16384_D8192_G8", "gated_norm_train", "bf16", 1, 16384, 8192, groups=8, gate="silu"),
        # training, every head of 64 normed before its gate, added to the residual with a learned scale; odd length
        norm_case("gated_norm_train_L1999_D4096_G64", "gated_norm_train", "f32", 1, 1999, 4096, groups=64, residual="io", scale="vector",
                  gate="sigmoid", norm_first=True),
        # a short odd prompt on a narrow layer
        recur_case("recur_L200_C256", "recur", "bf16", 1, 200, 256, "sigmoid", "complement", False),
        # seven prompts of uneven lengths packed in one row, each resumed from a state; x and both gates are slices of one projection
        recur_case("recur_varlen7_L16384_C4096", "recur", "bf16", 1, 16384, 4096, "decay", "unit", True, nseqs=7, initial=True, packed=True),
        # training in fp32 on packed documents, log decays given, odd sizes
        recur_case("recur_train_f32_L1999_C1000", "recur_train", "f32", 1, 1999, 1000, "log", "one", False, nseqs=5, initial=True),
        # training at the 16384-token layer's channels: the largest
        LARGEST,
        # one token of one sequence
        step_case("recur_step_B1_C8192", "bf16", 1, 1, 8192, "decay", "unit", True, 16),
        # four drafted tokens of a padded batch of 64 sequences, a few rows of it empty
        step_case("recur_step_B64_T4_C4096", "bf16", 64, 4, 4096, "decay", "unit", True, 80, holes=True),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["add_norm", "add_norm_train", "gated_norm", "gated_norm_train", "recur", "recur", "recur_train", "recur_train", "recur_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    batch = rng.choice([1, 1, 2, 5])
    if kind.endswith("norm") or kind.startswith(("add_norm", "gated_norm")):
        groups = 1 if kind.startswith("add") else rng.choice([1, 1, 2, 8, 64])
        width = groups * rng.choice([16, 64, 104, 128]) if groups > 8 else groups * rng.choice([64, 200, 512, 1000, 1024, 2560, 4096, 8192])
        width = min(width, 8192)
        residual = rng.choice(["none", "io", "f32"])
        c = norm_case("", kind, dtype, batch, log_int(rng, 1, 16384 // batch), width, groups, rng.choice(["rms", "rms", "layer"]),
                      residual, rng.choice(["none", "float", "vector"]), rng.random() < 0.3)
        if kind.startswith("gated"):
            c.update(gate=rng.choice(["silu", "silu", "sigmoid", "none"]), norm_first=rng.random() < 0.4)
    else:
        channels = rng.choice([64, 256, 1000, 2048, 2560, 4096, 8192])
        gate, scale = rng.choice(["log", "sigmoid", "decay", "decay"]), rng.choice(["one", "complement", "unit"])
        if kind == "recur_step":
            batch = log_int(rng, 1, 128)
            c = step_case("", dtype, batch, rng.choice([1, 1, 1, 2, 5]), channels, gate, scale, rng.random() < 0.5,
                          batch + rng.randint(1, 16), rng.random() < 0.5)
        else:
            nseqs = 0
            if rng.random() < 0.4:
                batch, nseqs = 1, rng.randint(2, 9)
            c = recur_case("", kind, dtype, batch, log_int(rng, 1 if not nseqs else 40, 16384 // batch), channels, gate, scale,
                           rng.random() < 0.5, nseqs, rng.random() < 0.5, rng.random() < 0.3)
    most = work(LARGEST)["bytes"]
    while work(c)["bytes"] > most:
        c["seqlen"] = c["seqlen"] * 2 // 3
    return {k: v for k, v in c.items() if k != "name"}


def work(c):
    size = 2 if c["dtype"] == "bf16" else 4
    tokens = c["batch"] * c["seqlen"]
    if "width" in c:
        n = tokens * c["width"]
        rsize = {"none": 0, "io": size, "f32": 4}[c["residual"]]
        gate = size if c["gate"] != "none" else 0
        if c["kind"].startswith("add"):
            # x and the residual read, y and the new residual written; for gradients dy and dr' read, dx and the residual's written
            out = rsize or size
            fwd, bwd = 2 * size + rsize + out, 2 * size + out + rsize
        else:
            # x, z and the residual read, the result written; for gradients dout read, dx and dz written (the residual's is dout)
            out = rsize or size
            fwd, bwd = size + gate + rsize + out, out + size + gate
        train = c["kind"].endswith("train")
        return {"bytes": n * (fwd + (bwd if train else 0)), "flops": n * (40 if train else 12)}
    ch = c["channels"]
    n = tokens * ch
    gsize = 4 if c["gate"] == "log" else size
    isize = size if c["in_gate"] else 0
    if c["kind"] == "recur_step":
        live = c["batch"] - (c["batch"] // 9 if c["holes"] else 0)
        return {"bytes": live * ch * 8 + live * c["seqlen"] * ch * (2 * size + gsize + isize), "flops": n * 20}
    seqs = c["nseqs"] or c["batch"]
    states = seqs * ch * 4
    # x, the gates and the initial states read, y and the final states written; for gradients dy read, dx and the gates' written
    fwd = n * (2 * size + gsize + isize) + states * (2 if c["initial"] else 1)
    bwd = n * (2 * size + gsize + isize) + states * (1 if c["initial"] else 0)
    train = c["kind"] == "recur_train"
    return {"bytes": fwd + (bwd if train else 0), "flops": n * (60 if train else 20)}


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def lengths_of(c, seed):
    """The packed sequences' lengths: uneven, one token at least, the case's tokens in all."""
    n, gen = c["nseqs"], torch.Generator().manual_seed(int(seed) + 1)
    cuts = torch.randperm(c["seqlen"] - 1, generator=gen)[: n - 1].sort().values.tolist()
    edges = [0] + [x + 1 for x in cuts] + [c["seqlen"]]
    return [edges[i + 1] - edges[i] for i in range(n)]


def prepare(c, seed):
    gen, io = generator(seed), IO[c["dtype"]]
    rn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    s = {"case": c}
    if "width" in c:
        b, L, D = c["batch"], c["seqlen"], c["width"]
        out = {"none": io, "io": io, "f32": torch.float32}[c["residual"]]
        s["x"] = rn(b, L, D).to(io)
        s["z"] = rn(b, L, D).to(io) if c["gate"] != "none" else None
        s["residual"] = (2 * rn(b, L, D)).to(out) if c["residual"] != "none" else None
        s["weight"] = 1 + 0.1 * rn(D)
        s["bias"] = 0.1 * rn(D) if c["bias"] else None
        s["scale"] = {"none": 1.0, "float": ALPHA}.get(c["scale"])
        if s["scale"] is None:
            s["scale"] = 0.5 + 0.1 * rn(D)
        if c["kind"].endswith("train"):
            if c["kind"].startswith("add"):
                s["dout"] = [rn(b, L, D).to(io), rn(b, L, D).to(out)]
            else:
                s["dout"] = [rn(b, L, D).to(out)]
            s["leaves"] = [t.requires_grad_(True) for t in (s["x"], s["z"], s["residual"], s["weight"], s["bias"], s["scale"])
                           if isinstance(t, torch.Tensor)]
        return s
    b, L, C = c["batch"], c["seqlen"], c["channels"]
    x = rn(b, L, C).to(io)
    if c["gate"] == "log":
        g = -torch.nn.functional.softplus(1.5 * rn(b, L, C) - 3.0)
    else:
        g = (rn(b, L, C) + (2.0 if c["gate"] == "sigmoid" else 0.0)).to(io)
    i = rn(b, L, C).to(io) if c["in_gate"] else None
    s["decay"] = 8.0 * torch.log(0.9 + 0.099 * torch.rand((C,), generator=gen, device="cuda")) if c["gate"] == "decay" else None
    s.update(x=x, g=g, in_gate=i)
    if c["kind"] == "recur_step":
        s["states"] = rn(c["slots"], C)
        index = torch.randperm(c["slots"], generator=gen, device="cuda")[:b].to(torch.int32)
        if c["holes"]:
            index[torch.randperm(b, generator=gen, device="cuda")[: b // 9]] = -1
        s["state_indices"] = index.contiguous()
        return s
    if c["packed"]:  # slices of one row of channels, as they leave a projection
        names = [k for k in ("x", "g", "in_gate") if s[k] is not None and s[k].dtype == io]
        row = torch.cat([s[k] for k in names], dim=-1).contiguous()
        for j, k in enumerate(names):
            s[k] = row[..., j * C: (j + 1) * C]
    s["nseqs"] = c["nseqs"] or b
    s["lengths"] = lengths_of(c, seed) if c["nseqs"] else None
    s["seq_idx"] = None
    if c["nseqs"]:
        s["seq_idx"] = torch.repeat_interleave(torch.arange(c["nseqs"], dtype=torch.int32), torch.tensor(s["lengths"])).reshape(1, L).cuda()
    s["initial_states"] = rn(s["nseqs"], C) if c["initial"] else None
    if c["kind"] == "recur_train":
        s["dy"] = rn(b, L, C).to(io)
        for k in ("x", "g", "in_gate", "decay", "initial_states"):
            if s[k] is not None:
                s[k] = s[k].detach().requires_grad_(True)
        s["leaves"] = [s[k] for k in ("x", "g", "in_gate", "decay", "initial_states") if s[k] is not None]
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def plain_unit(u, norm, groups):
    """u normed over each group of its last axis."""
    u = u.unflatten(-1, (groups, -1))
    if norm == "layer":
        u = u - u.mean(-1, keepdim=True)
    return (u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)).flatten(-2)


def plain_act(z, gate):
    return z * torch.sigmoid(z) if gate == "silu" else torch.sigmoid(z)


def plain_add_norm(s):
    c, x = s["case"], s["x"]
    r = x.float() * s["scale"]
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = plain_unit(r, c["norm"], 1) * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return [y.to(x.dtype), r.to(x.dtype if s["residual"] is None else s["residual"].dtype)]


def plain_gated_norm(s):
    c, x = s["case"], s["x"]
    act = plain_act(s["z"].float(), c["gate"]) if s["z"] is not None else None
    u = x.float()
    if act is not None and not c["norm_first"]:
        u = u * act
    n = plain_unit(u, c["norm"], c["groups"]) * s["weight"]
    if s["bias"] is not None:
        n = n + s["bias"]
    if act is not None and c["norm_first"]:
        n = n * act
    n = n * s["scale"]
    if s["residual"] is not None:
        return [(n + s["residual"].float()).to(s["residual"].dtype)]
    return [n.to(x.dtype)]


def plain_gates(x, g, i, decay, gate, input_scale):
    """(a, m u) of every row, in 32 bits."""
    g, u = g.float(), x.float()
    if i is not None:
        u = u * torch.sigmoid(i.float())
    if gate == "sigmoid":
        a, rest = torch.sigmoid(g), torch.sigmoid(-g)   # a and 1 - a
        square = rest * (1 + a)
    else:
        la = g if gate == "log" else decay * torch.sigmoid(g)
        a, rest, square = la.exp(), -torch.expm1(la), -torch.expm1(2 * la)
    if input_scale == "complement":
        u = u * rest
    elif input_scale == "unit":
        u = u * square.sqrt()
    return a, u


SPAN = 128


def plain_scan(a, b):
    """h_t = a_t h_{t-1} + b_t down (rows, channels), h before the first row zero: every span of rows by itself, then
    the state that enters each span, then what is left of it at each row."""
    rows = a.shape[0]
    pad = -rows % SPAN
    if pad:
        a, b = torch.cat([a, a.new_ones((pad, a.shape[1]))]), torch.cat([b, b.new_zeros((pad, b.shape[1]))])
    a, b = a.unflatten(0, (-1, SPAN)), b.unflatten(0, (-1, SPAN))
    own_h, left = [b[:, 0]], [a[:, 0]]
    for t in range(1, SPAN):
        own_h.append(a[:, t] * own_h[-1] + b[:, t])
        left.append(a[:, t] * left[-1])
    enter = [torch.zeros_like(b[0, 0])]
    for k in range(a.shape[0] - 1):
        enter.append(left[-1][k] * enter[-1] + own_h[-1][k])
    h = torch.stack(own_h, 1) + torch.stack(left, 1) * torch.stack(enter)[:, None]
    return h.flatten(0, 1)[:rows]


def edges_of(s):
    """First and last rows of the sequences in the (batch * seqlen) rows."""
    c = s["case"]
    lengths = torch.tensor(s["lengths"] or [c["seqlen"]] * c["batch"], device="cuda")
    last = lengths.cumsum(0) - 1
    return last - lengths + 1, last


def plain_recur(s):
    c = s["case"]
    a, b = plain_gates(s["x"], s["g"], s["in_gate"], s["decay"], c["gate"], c["input_scale"])
    a, b = a.flatten(0, 1), b.flatten(0, 1)
    first, last = edges_of(s)
    if s["initial_states"] is not None:
        b = b.index_add(0, first, a[first] * s["initial_states"])
    h = plain_scan(a.index_fill(0, first, 0.0), b)
    return h.reshape(s["x"].shape).to(s["x"].dtype), h[last]


def plain_step(s):
    c = s["case"]
    a, b = plain_gates(s["x"], s["g"], s["in_gate"], s["decay"], c["gate"], c["input_scale"])
    live = s["state_indices"] >= 0
    at = s["state_indices"].clamp(min=0).long()
    h, out = s["states"][at], []
    for t in range(c["seqlen"]):
        h = a[:, t] * h + b[:, t]
        out.append(h)
    s["states"][at[live]] = h[live]
    return torch.where(live[:, None, None], torch.stack(out, 1), 0.0).to(s["x"].dtype), s["states"]


def run(s):
    c = s["case"]
    kind = c["kind"]
    if "width" in c:
        if own:
            from state_space_model_mamba_amd import block_norm
            if kind == "add_norm":
                out = list(block_norm.add_norm_fwd(s["x"], s["residual"], s["weight"], s["bias"], s["scale"], eps=EPS, norm=c["norm"]))
            elif kind == "add_norm_train":
                out = list(block_norm.add_norm(s["x"], s["residual"], s["weight"], s["bias"], s["scale"], eps=EPS, norm=c["norm"]))
            else:
                call = block_norm.gated_norm if kind == "gated_norm_train" else block_norm.gated_norm_fwd
                out = [call(s["x"], s["z"], s["weight"], s["bias"], s["residual"], s["scale"], groups=c["groups"], eps=EPS, norm=c["norm"],
                            gate="silu" if c["gate"] == "none" else c["gate"], norm_before_gate=c["norm_first"])]
        else:
            out = plain_add_norm(s) if kind.startswith("add") else plain_gated_norm(s)
        if kind.endswith("train"):
            return {"out": out, "grads": torch.autograd.grad(out, s["leaves"], s["dout"])}
        return {"out": out}
    if own:
        from state_space_model_mamba_amd import recurrence
        more = dict(gate=c["gate"], input_scale=c["input_scale"])
        if kind == "recur_step":
            y = recurrence.linrec_step(s["x"], s["g"], s["states"], s["in_gate"], s["decay"], s["state_indices"], **more)
            return {"y": y, "states": s["states"]}
        if kind == "recur":
            r = recurrence.linrec_fwd(s["x"], s["g"], s["in_gate"], s["decay"], s["initial_states"], s["seq_idx"], nseqs=s["nseqs"],
                                      want_final_states=True, **more)
            return {"y": r["y"], "final_states": r["final_states"]}
        y, final = recurrence.linear_recurrence(s["x"], s["g"], s["in_gate"], s["decay"], s["initial_states"], s["seq_idx"], nseqs=s["nseqs"], **more)
    elif kind == "recur_step":
        y, states = plain_step(s)
        return {"y": y, "states": states}
    else:
        y, final = plain_recur(s)
        if kind == "recur":
            return {"y": y, "final_states": final}
    return {"y": y, "final_states": final.detach(), "grads": torch.autograd.grad(y, s["leaves"], s["dy"])}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, the gradients from their formulas
# ---------------------------------------------------------------------------------------------
def f64(t):
    return t.detach().double() if isinstance(t, torch.Tensor) else t


def exact_unit(u, norm, groups):
    """(u normed, the function that takes a gradient back through it)"""
    shape = u.shape
    v = u.reshape(shape[:-1] + (groups, shape[-1] // groups))
    if norm == "layer":
        v = v - v.sum(-1, keepdim=True) / v.shape[-1]
    r = ((v ** 2).sum(-1, keepdim=True) / v.shape[-1] + EPS) ** -0.5
    hat = v * r

    def back(d):
        d = d.reshape(v.shape)
        du = d - hat * (d * hat).sum(-1, keepdim=True) / v.shape[-1]
        if norm == "layer":
            du = du - d.sum(-1, keepdim=True) / v.shape[-1]
        return (r * du).reshape(shape)

    return hat.reshape(shape), back


def exact_norm(c, s):
    x, z, residual, w, b, scale = (f64(s[k]) for k in ("x", "z", "residual", "weight", "bias", "scale"))
    dout = [f64(t) for t in s.get("dout", [])]
    zero = 0.0 if b is None else b
    rows = (0, 1)
    if c["kind"].startswith("add"):
        r = x * scale + (0.0 if residual is None else residual)
        hat, back = exact_unit(r, c["norm"], 1)
        result = {"out": [hat * w + zero, r]}
        if dout:
            dr = dout[1] + back(dout[0] * w)
            grads = [dr * scale]
            if residual is not None:
                grads.append(dr)
            grads.append((dout[0] * hat).sum(rows))
            if b is not None:
                grads.append(dout[0].sum(rows))
            if c["scale"] == "vector":
                grads.append((dr * x).sum(rows))
            result["grads"] = grads
        return result
    one = torch.ones((), dtype=torch.float64, device=x.device)
    act, slope = one, None
    if z is not None:
        sg = 1 / (1 + (-z).exp())
        act, slope = (z * sg, sg * (1 + z * (1 - sg))) if c["gate"] == "silu" else (sg, sg * (1 - sg))
    before, after = (one, act) if c["norm_first"] else (act, one)
    hat, back = exact_unit(x * before, c["norm"], c["groups"])
    n = hat * w + zero
    result = {"out": [scale * n * after + (0.0 if residual is None else residual)]}
    if dout:
        d = dout[0] * scale
        dn = d * after
        du = back(dn * w)
        grads = [du * before]
        if z is not None:
            grads.append((d * n if c["norm_first"] else du * x) * slope)
        if residual is not None:
            grads.append(dout[0])
        grads.append((dn * hat).sum(rows))
        if b is not None:
            grads.append(dn.sum(rows))
        if c["scale"] == "vector":
            grads.append((dout[0] * n * after).sum(rows))
        result["grads"] = grads
    return result


def exact_gates(c, x, g, i, decay):
    """Of every row: the log decay and its derivative by g, m and its derivative by the log decay, sigmoid(i)."""
    sg = 1 / (1 + (-g).exp())
    if c["gate"] == "log":
        la, dla = g, torch.ones_like(g)
    elif c["gate"] == "sigmoid":
        la, dla = -torch.log1p((-g).exp()), 1 - sg
    else:
        la, dla = decay * sg, decay * sg * (1 - sg)
    a = la.exp()
    if c["input_scale"] == "one":
        m, dm = torch.ones_like(a), torch.zeros_like(a)
    elif c["input_scale"] == "complement":
        m, dm = -torch.expm1(la), -a
    else:
        m = (-torch.expm1(2 * la)).sqrt()
        dm = -a * a / m
    return a, sg, dla, m, dm, (None if i is None else 1 / (1 + (-i).exp()))


def exact(c, seed):
    s = prepare(c, seed)
    if "width" in c:
        return exact_norm(c, s)
    x, g, i, decay = (f64(s[k]) for k in ("x", "g", "in_gate", "decay"))
    a, sg, dla, m, dm, si = exact_gates(c, x, g, i, decay)
    gated = x if si is None else x * si
    if c["kind"] == "recur_step":
        states = s["states"].double()
        y = torch.zeros_like(x)
        for row, at in enumerate(s["state_indices"].tolist()):
            if at >= 0:
                for t in range(c["seqlen"]):
                    states[at] = a[row, t] * states[at] + m[row, t] * gated[row, t]
                    y[row, t] = states[at]
        return {"y": y, "states": states}
    rows = c["batch"] * c["seqlen"]
    flat = lambda t: t.reshape(rows, c["channels"])  # noqa: E731
    af, bf = flat(a), flat(m * gated)
    first, last = (t.tolist() for t in edges_of(s))
    h0 = f64(s["initial_states"]) if c["initial"] else torch.zeros((len(first), c["channels"]), dtype=torch.float64, device=x.device)
    h, before = torch.empty_like(af), torch.empty_like(af)
    for q, (lo, hi) in enumerate(zip(first, last)):
        state = h0[q]
        for t in range(lo, hi + 1):
            before[t] = state
            state = torch.addcmul(bf[t], af[t], state)
            h[t] = state
    result = {"y": h.reshape(x.shape), "final_states": h[last]}
    if c["kind"] == "recur":
        return result
    # the gradient of h_t: its own, and a_{t+1} times the next row's
    e, dh0 = flat(f64(s["dy"])).clone(), torch.empty_like(h0)
    for q, (lo, hi) in enumerate(zip(first, last)):
        for t in range(hi - 1, lo - 1, -1):
            e[t].addcmul_(af[t + 1], e[t + 1])
        dh0[q] = af[lo] * e[lo]
    e = e.reshape(x.shape)
    dlog = e * (a * before.reshape(x.shape) + dm * gated)   # by the log decay
    du = e * m
    grads = [du if si is None else du * si, dlog * dla]
    if si is not None:
        grads.append(du * x * si * (1 - si))
    if decay is not None:
        grads.append((dlog * sg).sum((0, 1)))
    if c["initial"]:
        grads.append(dh0)
    result["grads"] = grads
    return result
