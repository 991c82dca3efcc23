"""ctypes binding of the gated delta rule of libssd_bwd.so (include/gated_delta.h).

Argument marshalling only, as in ``ssd``: shapes and dtypes are checked,
outputs and the workspace are allocated with torch on the inputs' device, and
the C entry point is called on that device's current HIP stream.  Every
arithmetic step runs in the library's kernels; the calls raise if the library
is missing or returns an error.

``delta_fwd`` / ``delta_bwd`` run whole sequences, ``gated_delta_rule`` pairs
them as an autograd function, ``delta_step`` runs few tokens on a pool of
states kept in memory (the states that ``delta_fwd`` returns have its layout).
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from state_space_model_mamba_amd import ssd

EXPORTED = ("delta_fwd", "delta_bwd", "delta_step", "delta_workspace_size")
MAX_STEP_TOKENS = 64


class DeltaShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("batch", "seqlen", "nheads", "headdim", "ngroups", "dstate", "nseqs",
                                               "q_batch_stride", "q_row_stride", "k_batch_stride", "k_row_stride",
                                               "v_batch_stride", "v_row_stride")] +
                [("scale", ctypes.c_float), ("io_dtype", ctypes.c_int32)])


_lib = None


def load_library():
    """The shared library with the delta entry points' argument types set (raises if it is not built)."""
    global _lib
    if _lib is None:
        lib = ssd.load_library()
        vp, sp, n = ctypes.c_void_p, ctypes.POINTER(DeltaShape), ctypes.c_size_t
        lib.delta_workspace_size.restype = ctypes.c_int
        lib.delta_workspace_size.argtypes = [sp, ctypes.c_int, ctypes.POINTER(n)]
        lib.delta_fwd.restype = ctypes.c_int
        lib.delta_fwd.argtypes = [sp] + [vp] * 10 + [n, vp]
        lib.delta_bwd.restype = ctypes.c_int
        lib.delta_bwd.argtypes = [sp] + [vp] * 16 + [n, vp]
        lib.delta_step.restype = ctypes.c_int
        lib.delta_step.argtypes = [sp] + [vp] * 6 + [ctypes.c_int64] + [vp] * 3
        _lib = lib
    return _lib


def make_shape(batch, seqlen, nheads, headdim, ngroups, dstate, nseqs, io_dtype=ssd.SSD_IO_BF16, scale=None,
               strides=(0, 0, 0, 0, 0, 0)) -> DeltaShape:
    scale = 1.0 / math.sqrt(dstate) if scale is None else float(scale)
    return DeltaShape(batch, seqlen, nheads, headdim, ngroups, dstate, nseqs, *strides, scale, io_dtype)


def workspace_size(shape: DeltaShape, backward: bool = False) -> int:
    """Bytes of workspace delta_fwd, or with ``backward`` delta_bwd, needs."""
    n = ctypes.c_size_t(0)
    rc = load_library().delta_workspace_size(ctypes.byref(shape), int(bool(backward)), ctypes.byref(n))
    if rc:
        raise ssd.SsdError(rc, "delta_workspace_size")
    return n.value


@functools.lru_cache(maxsize=256)
def _sized(batch, seqlen, nheads, headdim, ngroups, dstate, nseqs, io_dtype, scale, strides) -> DeltaShape:
    """make_shape, kept per sizes (callers read it only)."""
    return make_shape(batch, seqlen, nheads, headdim, ngroups, dstate, nseqs, io_dtype, scale, strides)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, nseqs, io_dtype, backward) -> int:
    return workspace_size(make_shape(batch, seqlen, nheads, headdim, ngroups, dstate, nseqs, io_dtype), backward)


def row_strides(t, name):
    """(batch, row) strides of a (batch, rows, heads, width) tensor whose last two axes are contiguous."""
    if t.is_contiguous():
        return 0, 0
    b, L, n, w = t.shape
    sb, sl, sn, sw = t.stride()
    if (sw != 1 and w > 1) or (sn != w and n > 1):
        raise ValueError(f"{name} must be contiguous in its last two axes")
    if L == 1:
        sl = n * w
    if b == 1:
        sb = L * sl
    if sb == 0 and sl == 0:
        raise ValueError(f"{name} may be broadcast over batch or rows, not over both")
    return sb, sl


def _check_strided(t, name, dtype, shape, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return row_strides(t, name)


def _gradient(t):
    """An incoming gradient as the kernels read it: contiguous, from an address of 16 bytes (a slice of a larger
    gradient may start anywhere)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


class _on:
    """The device of the tensors made current (the library launches on the current device)."""
    __slots__ = ("prev", "index")

    def __init__(self, device):
        self.index = device.index

    def __enter__(self):
        self.prev = torch.cuda.current_device()
        if self.prev != self.index:
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        if self.prev != self.index:
            torch.cuda.set_device(self.prev)


def _inputs(what, q, k, v, g, beta, nseqs, scale) -> DeltaShape:
    dev, io = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on a HIP device; got tensors on {dev}")
    if io not in (torch.bfloat16, torch.float32):
        raise ValueError(f"unsupported io dtype {io}")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v are (batch, seqlen, heads, width)")
    b, L, G, N = q.shape
    H, P = v.shape[2], v.shape[3]
    strides = (*_check_strided(q, "q", io, (b, L, G, N), dev), *_check_strided(k, "k", io, (b, L, G, N), dev),
               *_check_strided(v, "v", io, (b, L, H, P), dev))
    ssd._check(g, "g", torch.float32, (b, L, H), dev)
    ssd._check(beta, "beta", torch.float32, (b, L, H), dev)
    return _sized(b, L, H, P, G, N, nseqs, ssd.SSD_IO_BF16 if io == torch.bfloat16 else ssd.SSD_IO_F32,
                  None if scale is None else float(scale), strides)


def _copy(shape: DeltaShape) -> DeltaShape:
    """A shape for the caller to keep (_sized's is shared by all calls of its sizes)."""
    return DeltaShape.from_buffer_copy(shape)


def _nseqs(q, initial_states, seq_idx, nseqs) -> int:
    if initial_states is not None:
        if nseqs is not None and nseqs != initial_states.shape[0]:
            raise ValueError(f"nseqs is {nseqs}, initial_states holds {initial_states.shape[0]}")
        return initial_states.shape[0]
    if seq_idx is None:
        if nseqs is not None and nseqs != q.shape[0]:
            raise ValueError(f"nseqs is {nseqs}; without seq_idx every batch row is one sequence")
        return q.shape[0]
    if nseqs is None:
        raise ValueError("pass nseqs (number of sequence starts) with seq_idx")
    return int(nseqs)


def _workspace(shape, backward, workspace, dev):
    nbytes = _workspace_bytes(shape.batch, shape.seqlen, shape.nheads, shape.headdim, shape.ngroups, shape.dstate,
                              shape.nseqs, shape.io_dtype, backward)
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return workspace


def delta_fwd(q, k, v, g, beta, initial_states=None, seq_idx=None, scale: Optional[float] = None,
              nseqs: Optional[int] = None, want_final_states: bool = False,
              workspace: Optional[torch.Tensor] = None) -> dict:
    """The gated delta rule over whole sequences (the recurrence of include/gated_delta.h).

    q, k: (b, L, G, N) and v: (b, L, H, P) in bf16 or fp32 (one dtype; slices of wider rows are taken as they
    are), g (log decay) and beta: (b, L, H) fp32, initial_states: (S, H, P, N) fp32 or None, seq_idx: (b, L) int32
    or None.  ``nseqs`` is needed only when seq_idx is given without initial_states; ``scale`` is 1 / sqrt(N) by
    default.  Returns a dict with o (like v, contiguous) and final_states ((S, H, P, N) fp32, or None).
    """
    S = _nseqs(q, initial_states, seq_idx, nseqs)
    shape = _inputs("delta_fwd", q, k, v, g, beta, S, scale)
    dev = q.device
    b, L, H, P, N = shape.batch, shape.seqlen, shape.nheads, shape.headdim, shape.dstate
    ssd._check(initial_states, "initial_states", torch.float32, (S, H, P, N), dev)
    ssd._check(seq_idx, "seq_idx", torch.int32, (b, L), dev)
    workspace = _workspace(shape, False, workspace, dev)
    o = torch.empty((b, L, H, P), dtype=v.dtype, device=dev)
    final = torch.empty((S, H, P, N), dtype=torch.float32, device=dev) if want_final_states else None
    lib = load_library()
    with _on(dev):
        rc = lib.delta_fwd(ctypes.byref(shape), ssd._ptr(q), ssd._ptr(k), ssd._ptr(v), ssd._ptr(g), ssd._ptr(beta),
                           ssd._ptr(initial_states), ssd._ptr(seq_idx), ssd._ptr(o), ssd._ptr(final),
                           ssd._ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(dev))
    if rc:
        raise ssd.SsdError(rc, "delta_fwd")
    return {"o": o, "final_states": final, "workspace": workspace, "shape": _copy(shape)}


def delta_bwd(q, k, v, g, beta, do, initial_states=None, seq_idx=None, d_final_states=None,
              scale: Optional[float] = None, nseqs: Optional[int] = None, want_d_initial_states: bool = True,
              workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of sum(do * o) + sum(d_final_states * final_states) of delta_fwd, from its inputs.

    Returns a dict with dq, dk, dv (io dtype, contiguous), dg, dbeta (fp32) and d_initial_states ((S, H, P, N) fp32,
    or None).
    """
    S = _nseqs(q, initial_states, seq_idx, nseqs)
    shape = _inputs("delta_bwd", q, k, v, g, beta, S, scale)
    dev = q.device
    b, L, H, P, G, N = shape.batch, shape.seqlen, shape.nheads, shape.headdim, shape.ngroups, shape.dstate
    ssd._check(do, "do", v.dtype, (b, L, H, P), dev)
    ssd._check(initial_states, "initial_states", torch.float32, (S, H, P, N), dev)
    ssd._check(d_final_states, "d_final_states", torch.float32, (S, H, P, N), dev)
    ssd._check(seq_idx, "seq_idx", torch.int32, (b, L), dev)
    workspace = _workspace(shape, True, workspace, dev)
    out = {"dq": torch.empty((b, L, G, N), dtype=q.dtype, device=dev),
           "dk": torch.empty((b, L, G, N), dtype=q.dtype, device=dev),
           "dv": torch.empty((b, L, H, P), dtype=q.dtype, device=dev),
           "dg": torch.empty((b, L, H), dtype=torch.float32, device=dev),
           "dbeta": torch.empty((b, L, H), dtype=torch.float32, device=dev),
           "d_initial_states": (torch.empty((S, H, P, N), dtype=torch.float32, device=dev)
                                if want_d_initial_states else None)}
    lib = load_library()
    with _on(dev):
        rc = lib.delta_bwd(ctypes.byref(shape), ssd._ptr(q), ssd._ptr(k), ssd._ptr(v), ssd._ptr(g), ssd._ptr(beta),
                           ssd._ptr(initial_states), ssd._ptr(seq_idx), ssd._ptr(do), ssd._ptr(d_final_states),
                           ssd._ptr(out["dq"]), ssd._ptr(out["dk"]), ssd._ptr(out["dv"]), ssd._ptr(out["dg"]),
                           ssd._ptr(out["dbeta"]), ssd._ptr(out["d_initial_states"]), ssd._ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(dev))
    if rc:
        raise ssd.SsdError(rc, "delta_bwd")
    out["workspace"] = workspace
    out["shape"] = _copy(shape)
    return out


class GatedDeltaRule(torch.autograd.Function):
    """delta_fwd paired with delta_bwd, which recomputes the states from the saved inputs: nothing but the
    inputs is kept between the two."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, initial_states, seq_idx, scale, nseqs):
        ctx.set_materialize_grads(False)
        scale = None if scale is None else float(scale)   # the backward's too, whatever a tensor holds by then
        r = delta_fwd(q, k, v, g, beta, initial_states, seq_idx, scale, nseqs, want_final_states=True)
        ctx.save_for_backward(q, k, v, g, beta, initial_states, seq_idx)
        ctx.scale, ctx.nseqs = scale, nseqs
        return r["o"], r["final_states"]

    @staticmethod
    @once_differentiable
    def backward(ctx, do, d_final):
        q, k, v, g, beta, h0, seq_idx = ctx.saved_tensors
        if do is None and d_final is None:
            return (None,) * 9
        do = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if do is None else _gradient(do)
        want_h0 = h0 is not None and ctx.needs_input_grad[5]
        r = delta_bwd(q, k, v, g, beta, do, h0, seq_idx, None if d_final is None else _gradient(d_final), ctx.scale,
                      ctx.nseqs, want_d_initial_states=want_h0)
        return r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], r["d_initial_states"], None, None, None


def gated_delta_rule(q, k, v, g, beta, initial_states=None, seq_idx=None, scale: Optional[float] = None,
                     nseqs: Optional[int] = None):
    """(o, final_states) of delta_fwd with autograd support: gradients reach q, k, v, g, beta and initial_states,
    from o and from final_states."""
    return GatedDeltaRule.apply(q, k, v, g, beta, initial_states, seq_idx, scale, nseqs)


def delta_step(q, k, v, g, beta, states, state_indices=None, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The recurrence for T = q.shape[1] tokens (1 .. 64) of each of b sequences, on a pool of states.

    q, k: (b, T, G, N), v: (b, T, H, P), g, beta: (b, T, H) as for delta_fwd; states: (slots, H, P, N) fp32,
    updated in place; state_indices: (b) int32, the state of each row (None: row b has state b).  A row whose index
    is negative (or past the pool) is empty: its o is zero.  Rows that name the same state take their turns in row
    order.  Returns o (like v, contiguous; ``out`` when given).  Not differentiable; autograd sees that states (and
    out) change.
    """
    shape = _inputs("delta_step", q, k, v, g, beta, q.shape[0], scale)
    dev = q.device
    b, T, H, P, N = shape.batch, shape.seqlen, shape.nheads, shape.headdim, shape.dstate
    if T > MAX_STEP_TOKENS:
        raise ValueError(f"delta_step takes up to {MAX_STEP_TOKENS} tokens a row; got {T} (use delta_fwd)")
    if states.dim() != 4:
        raise ValueError("states is (slots, heads, headdim, dstate)")
    ssd._check(states, "states", torch.float32, (states.shape[0], H, P, N), dev)
    if state_indices is None:
        if states.shape[0] < b:
            raise ValueError(f"states holds {states.shape[0]} states for {b} rows")
    else:
        ssd._check(state_indices, "state_indices", torch.int32, (b,), dev)
    if out is None:
        out = torch.empty((b, T, H, P), dtype=v.dtype, device=dev)
    else:
        ssd._check(out, "out", v.dtype, (b, T, H, P), dev)
    lib = load_library()
    with _on(dev):
        rc = lib.delta_step(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                            beta.data_ptr(), states.data_ptr(), states.shape[0],
                            None if state_indices is None else state_indices.data_ptr(), out.data_ptr(),
                            _stream(dev))
    if rc:
        raise ssd.SsdError(rc, "delta_step")
    for t in (states, out):
        if not t.is_inference():
            torch.autograd.graph.increment_version(t)
    return out
