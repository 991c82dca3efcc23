"""Host-side checks of the C ABIs of the gated delta rule and of the q/k norm
(include/gated_delta.h, include/qk_norm.h) and of their bindings: no GPU
needed, nothing is launched.  Bad arguments come back as status codes or
exceptions before any work is enqueued."""
import ctypes
import os
import re

import pytest
import torch

from state_space_model_mamba_amd import delta, qk_norm, ssd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
vp = ctypes.c_void_p


def header_functions(name, prefix):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\**(%s\w+)\s*\(" % prefix, text, flags=re.M)))


@pytest.mark.parametrize("header,prefix,module", [("gated_delta.h", "delta_", delta), ("qk_norm.h", "qk_norm_", qk_norm)])
def test_library_exports_every_declared_function(header, prefix, module):
    lib = module.load_library()
    names = header_functions(header, prefix)
    assert set(names) == set(module.EXPORTED), names
    for n in names:
        assert hasattr(lib, n), n


BASE = dict(batch=2, seqlen=100, nheads=4, headdim=16, ngroups=2, dstate=32, nseqs=2)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), -2), (dict(seqlen=0), -2), (dict(nheads=5), -2), (dict(ngroups=0), -2), (dict(headdim=12), -2),
    (dict(headdim=1032), -2), (dict(dstate=20), -2), (dict(dstate=136), -2), (dict(io_dtype=3), -2), (dict(nseqs=0), -2),
    (dict(nheads=65538, ngroups=1), -2), (dict(batch=1 << 20, seqlen=1 << 12), -2), (dict(strides=(4, 0, 0, 0, 0, 0)), -2),
    (dict(strides=(0, 0, 0, 0, -8, 64)), -2), (dict(strides=(0, 0, 0, 1 << 27, 0, 0)), -2),
    (dict(nheads=65535, ngroups=1, headdim=1024), 0), (dict(nheads=65535, ngroups=65535, headdim=1032), -2),
])
def test_shapes_at_and_past_the_limits(kw, code):
    s = delta.make_shape(**{**BASE, **kw})
    n = ctypes.c_size_t(0)
    assert delta.load_library().delta_workspace_size(ctypes.byref(s), 0, ctypes.byref(n)) == code


def test_workspace_sizes_grow_with_the_problem():
    small, large = delta.make_shape(**BASE), delta.make_shape(**{**BASE, "seqlen": 1000})
    assert 0 < delta.workspace_size(small) < delta.workspace_size(small, backward=True)
    assert delta.workspace_size(small) < delta.workspace_size(large)
    assert delta.load_library().delta_workspace_size(ctypes.byref(small), 0, None) == -1


FAKE = {k: 0x100000 * (i + 1) for i, k in enumerate(
    ["q", "k", "v", "g", "beta", "h0", "seq", "o", "fin", "dout", "dfin", "dq", "dk", "dv", "dg", "db", "dh0", "ws", "states", "index"])}


def fwd(s, p, ws_bytes=1 << 40):
    return delta.load_library().delta_fwd(ctypes.byref(s), *[vp(p.get(n)) for n in ("q", "k", "v", "g", "beta", "h0", "seq", "o", "fin", "ws")],
                                          ctypes.c_size_t(ws_bytes), None)


def bwd(s, p, ws_bytes=1 << 40):
    return delta.load_library().delta_bwd(ctypes.byref(s), *[vp(p.get(n)) for n in (
        "q", "k", "v", "g", "beta", "h0", "seq", "dout", "dfin", "dq", "dk", "dv", "dg", "db", "dh0", "ws")], ctypes.c_size_t(ws_bytes), None)


def step(s, p, nslots=8):
    return delta.load_library().delta_step(ctypes.byref(s), *[vp(p.get(n)) for n in ("q", "k", "v", "g", "beta", "states")],
                                           nslots, vp(p.get("index")), vp(p.get("o")), None)


def test_delta_argument_errors_are_reported_before_launch():
    s = delta.make_shape(**BASE)
    few = delta.make_shape(**{**BASE, "seqlen": 4})
    for call, needed in ((fwd, ("q", "k", "v", "g", "beta", "o", "ws")),
                         (bwd, ("q", "k", "v", "g", "beta", "dout", "dq", "dk", "dv", "dg", "db", "ws")),
                         (step, ("q", "k", "v", "g", "beta", "states", "o"))):
        for missing in needed:
            p = dict(FAKE)
            p.pop(missing)
            assert call(few if call is step else s, p) == -1, (call.__name__, missing)
    for name in ("q", "k", "v", "h0", "o", "fin", "ws"):
        assert fwd(s, dict(FAKE, **{name: FAKE[name] + 8})) == -4, name
    for name in ("q", "v", "dout", "dfin", "dq", "dv", "dh0", "ws"):
        assert bwd(s, dict(FAKE, **{name: FAKE[name] + 4})) == -4, name
    assert fwd(s, FAKE, ws_bytes=64) == -3 and bwd(s, FAKE, ws_bytes=64) == -3
    assert fwd(s, dict(FAKE, o=FAKE["v"])) == -1
    assert bwd(s, dict(FAKE, dk=FAKE["k"])) == -1 and bwd(s, dict(FAKE, dv=FAKE["dout"])) == -1
    one = delta.make_shape(**{**BASE, "nseqs": 3})
    assert fwd(one, dict(FAKE, seq=None)) == -1   # without seq_idx every batch row is one sequence
    assert step(s, FAKE) == -2                    # 100 tokens
    assert step(few, FAKE, nslots=0) == -1
    assert step(few, dict(FAKE, index=None), nslots=1) == -1
    assert step(few, dict(FAKE, states=FAKE["states"] + 4)) == -4


def norm_shape(**kw):
    return qk_norm.make_shape(**{**dict(batch=2, seqlen=5, qheads=4, kheads=2, dstate=32, rot_dim=16), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), -2), (dict(qheads=0), -2), (dict(kheads=-1), -2), (dict(dstate=20), -2), (dict(dstate=264), -2), (dict(rot_dim=3), -2),
    (dict(rot_dim=34), -2), (dict(rot_dim=-2), -2), (dict(norm=2), -2), (dict(interleaved=2), -2), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(io_dtype=9), -2), (dict(strides=(3, 128, 0, 0)), -2),
])
def test_qk_norm_shapes_are_rejected(kw, code):
    n = ctypes.c_size_t(0)
    assert qk_norm.load_library().qk_norm_bwd_workspace_size(ctypes.byref(norm_shape(**kw)), ctypes.byref(n)) == code


def test_qk_norm_argument_errors_are_reported_before_launch():
    lib, a = qk_norm.load_library(), {n: 0x100000 * (i + 1) for i, n in enumerate("q k wq wk pos f oq ok dq dk ws dyq dyk".split())}

    def f(s, **kw):
        p = dict(a, **kw)
        return lib.qk_norm_fwd(ctypes.byref(s), *[vp(p[n]) for n in "q k wq wk pos f oq ok".split()], None)

    def b(s, ws_bytes=1 << 30, **kw):
        p = dict(a, **kw)
        return lib.qk_norm_bwd(ctypes.byref(s), *[vp(p[n]) for n in "q k wq wk pos f dyq dyk dq dk wq wk ws".split()], ctypes.c_size_t(ws_bytes), None)

    s = norm_shape()
    for name in ("q", "k", "f", "oq", "ok"):
        assert f(s, **{name: None}) == -1, name
    for name in ("q", "k", "f", "dyq", "dyk", "dq", "dk", "ws"):
        assert b(s, **{name: None}) == -1, name
    assert f(s, q=a["q"] + 2) == -4 and b(s, dk=a["dk"] + 8) == -4
    assert b(s, ws_bytes=8) == -3 and b(s, dq=a["q"]) == -1
    bad = norm_shape()
    bad.reserved = 1
    assert f(bad) == -1


def tensors(b=2, L=5, H=4, P=8, G=2, N=16, dev="cpu"):
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device=dev)  # noqa: E731
    return [z(b, L, G, N), z(b, L, G, N), z(b, L, H, P), z(b, L, H, d=torch.float32), z(b, L, H, d=torch.float32)]


def test_bindings_refuse_the_cpu_and_bad_arguments():
    t = tensors()
    with pytest.raises(ValueError, match="HIP device"):
        delta.delta_fwd(*t)
    with pytest.raises(ValueError, match="HIP device"):
        delta.delta_bwd(*t, t[2])
    with pytest.raises(ValueError, match="HIP device"):
        delta.delta_step(*t, torch.zeros(2, 4, 8, 16))
    with pytest.raises(ValueError, match="HIP device"):
        qk_norm.qk_norm_rope_fwd(t[0], t[1])
    with pytest.raises(ValueError, match="nseqs"):
        delta.delta_fwd(*t, seq_idx=torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="nseqs"):
        delta.delta_fwd(*t, nseqs=3)
    with pytest.raises(ValueError, match="nseqs"):
        delta.delta_fwd(*t, initial_states=torch.zeros(2, 4, 8, 16), nseqs=4)


def test_row_strides_of_slices():
    x = torch.zeros(3, 7, 4 * 16 + 2 * 8)
    s = x[..., 64:].unflatten(-1, (2, 8))
    assert delta.row_strides(x.unflatten(-1, (10, 8)), "x") == (0, 0)   # contiguous
    assert delta.row_strides(s, "s") == (7 * 80, 80)
    assert delta.row_strides(s[:1], "s") == (7 * 80, 80)
    assert delta.row_strides(s[:, :1], "s") == (7 * 80, 16)
    assert delta.row_strides(x[:1, :1, :16].unflatten(-1, (2, 8)).expand(3, 7, 2, 8)[:, :1], "s") == (0, 16)
    for bad in (s.transpose(2, 3), s[..., ::2], s[:, :, ::2].expand(3, 7, 2, 8)[..., :4]):
        with pytest.raises(ValueError, match="contiguous"):
            delta.row_strides(bad, "s")
    with pytest.raises(ValueError, match="broadcast"):
        delta.row_strides(x[:1, :1, :16].unflatten(-1, (2, 8)).expand(3, 7, 2, 8), "s")


def test_step_refuses_its_output_in_an_inputs_place():
    few = delta.make_shape(**{**BASE, "seqlen": 4})
    for name in ("q", "k", "v", "states"):
        assert step(few, dict(FAKE, o=FAKE[name])) == -1, name
