"""ctypes binding of the per-head q/k norm with rotation of libssd_bwd.so (include/qk_norm.h).

Argument marshalling only, as in ``ssd``; every arithmetic step runs in the
library's kernels, and the calls raise if the library is missing or returns
an error.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from state_space_model_mamba_amd import ssd
from state_space_model_mamba_amd.delta import _check_strided, _gradient, _on, _stream

QK_NORM_RMS, QK_NORM_L2 = 0, 1
NORMS = {"rms": QK_NORM_RMS, "l2": QK_NORM_L2}
EXPORTED = ("qk_norm_fwd", "qk_norm_bwd", "qk_norm_bwd_workspace_size")


class QkNormShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("batch", "seqlen", "qheads", "kheads", "dstate", "q_batch_stride",
                                               "q_row_stride", "k_batch_stride", "k_row_stride")] +
                [(n, ctypes.c_int32) for n in ("rot_dim", "interleaved", "norm", "io_dtype")] +
                [("eps", ctypes.c_float), ("reserved", ctypes.c_int32)])


_lib = None


def load_library():
    """The shared library with the qk_norm entry points' argument types set (raises if it is not built)."""
    global _lib
    if _lib is None:
        lib = ssd.load_library()
        vp, sp, n = ctypes.c_void_p, ctypes.POINTER(QkNormShape), ctypes.c_size_t
        lib.qk_norm_fwd.restype = ctypes.c_int
        lib.qk_norm_fwd.argtypes = [sp] + [vp] * 9
        lib.qk_norm_bwd_workspace_size.restype = ctypes.c_int
        lib.qk_norm_bwd_workspace_size.argtypes = [sp, ctypes.POINTER(n)]
        lib.qk_norm_bwd.restype = ctypes.c_int
        lib.qk_norm_bwd.argtypes = [sp] + [vp] * 13 + [n, vp]
        _lib = lib
    return _lib


def make_shape(batch, seqlen, qheads, kheads, dstate, rot_dim=0, interleaved=False, norm="rms",
               io_dtype=ssd.SSD_IO_BF16, eps=1e-6, strides=(0, 0, 0, 0)) -> QkNormShape:
    norm = NORMS[norm] if isinstance(norm, str) else int(norm)
    return QkNormShape(batch, seqlen, qheads, kheads, dstate, *strides, rot_dim, int(interleaved), norm, io_dtype, eps, 0)


def workspace_size(shape: QkNormShape) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().qk_norm_bwd_workspace_size(ctypes.byref(shape), ctypes.byref(n))
    if rc:
        raise ssd.SsdError(rc, "qk_norm_bwd_workspace_size")
    return n.value


@functools.lru_cache(maxsize=256)
def _sized(*sizes) -> tuple[QkNormShape, int]:
    """make_shape and its workspace size, kept per sizes (callers read them only)."""
    shape = make_shape(*sizes)
    return shape, workspace_size(shape)


def _shape(q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved) -> tuple[QkNormShape, int]:
    dev, io = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError(f"qk_norm_rope runs on a HIP device; got tensors on {dev}")
    if io not in (torch.bfloat16, torch.float32):
        raise ValueError(f"unsupported io dtype {io}")
    if norm not in NORMS:
        raise ValueError(f"norm is one of {sorted(NORMS)}; got {norm!r}")
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k are (batch, seqlen, heads, dstate)")
    b, L, Gq, N = q.shape
    strides = (*_check_strided(q, "q", io, (b, L, Gq, N), dev),
               *(_check_strided(k, "k", io, (b, L, k.shape[2], N), dev) if k is not None else (0, 0)))
    ssd._check(q_weight, "q_weight", torch.float32, (N,), dev)
    ssd._check(k_weight, "k_weight", torch.float32, (N,), dev)
    if k is None and k_weight is not None:
        raise ValueError("k_weight goes with k")
    ssd._check(positions, "positions", torch.int32, (b, L), dev)
    rot = 0
    if inv_freq is not None:
        ssd._check(inv_freq, "inv_freq", torch.float32, (inv_freq.numel(),), dev)
        rot = 2 * inv_freq.numel()
        if rot > N:
            raise ValueError(f"inv_freq turns {rot} values of rows of {N}")
    elif positions is not None:
        raise ValueError("positions go with inv_freq")
    return _sized(b, L, Gq, 0 if k is None else k.shape[2], N, rot, bool(interleaved), norm,
                  ssd.SSD_IO_BF16 if io == torch.bfloat16 else ssd.SSD_IO_F32, float(eps), strides)


def qk_norm_rope_fwd(q, k=None, q_weight=None, k_weight=None, positions=None, inv_freq=None, eps: float = 1e-6,
                     norm: str = "rms", interleaved: bool = False):
    """(q_out, k_out): every head of q (b, L, Gq, N) and k (b, L, Gk, N) normed, scaled by its weight (N) fp32 or
    None, and its first 2 * len(inv_freq) values turned by positions * inv_freq.

    q, k: bf16 or fp32 (slices of wider rows are taken as they are; k may be None, and k_out is then None);
    positions: (b, L) int32, or None for 0 .. L-1; inv_freq: fp32, or None for no rotation; norm: "rms"
    (1 / sqrt(mean x^2 + eps)) or "l2" (1 / sqrt(sum x^2 + eps)); interleaved: pairs (2j, 2j+1) instead of
    (j, j + len(inv_freq)).
    """
    shape, _ = _shape(q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved)
    dev = q.device
    q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    k_out = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=dev)
    lib = load_library()
    with _on(dev):
        rc = lib.qk_norm_fwd(ctypes.byref(shape), ssd._ptr(q), ssd._ptr(k), ssd._ptr(q_weight), ssd._ptr(k_weight),
                             ssd._ptr(positions), ssd._ptr(inv_freq), ssd._ptr(q_out), ssd._ptr(k_out),
                             _stream(dev))
    if rc:
        raise ssd.SsdError(rc, "qk_norm_fwd")
    return q_out, k_out


def qk_norm_rope_bwd(q, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out, eps: float = 1e-6,
                     norm: str = "rms", interleaved: bool = False, workspace: Optional[torch.Tensor] = None) -> dict:
    """dict of dq, dk (like q and k, contiguous), dq_weight and dk_weight ((N) fp32, or None without the weight)."""
    shape, nbytes = _shape(q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved)
    dev = q.device
    ssd._check(dq_out, "dq_out", q.dtype, tuple(q.shape), dev)
    if (k is None) != (dk_out is None):
        raise ValueError("dk_out goes with k")
    if k is not None:
        ssd._check(dk_out, "dk_out", k.dtype, tuple(k.shape), dev)
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    weight = lambda w: None if w is None else torch.empty(w.shape, dtype=torch.float32, device=dev)  # noqa: E731
    out = {"dq": torch.empty(q.shape, dtype=q.dtype, device=dev),
           "dk": None if k is None else torch.empty(k.shape, dtype=k.dtype, device=dev),
           "dq_weight": weight(q_weight), "dk_weight": weight(k_weight)}
    lib = load_library()
    with _on(dev):
        rc = lib.qk_norm_bwd(ctypes.byref(shape), ssd._ptr(q), ssd._ptr(k), ssd._ptr(q_weight), ssd._ptr(k_weight),
                             ssd._ptr(positions), ssd._ptr(inv_freq), ssd._ptr(dq_out), ssd._ptr(dk_out),
                             ssd._ptr(out["dq"]), ssd._ptr(out["dk"]), ssd._ptr(out["dq_weight"]),
                             ssd._ptr(out["dk_weight"]), ssd._ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(dev))
    if rc:
        raise ssd.SsdError(rc, "qk_norm_bwd")
    return out


class QkNormRope(torch.autograd.Function):
    """qk_norm_rope_fwd paired with qk_norm_rope_bwd (deterministic); only the inputs are kept between the two."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        ctx.args = (float(eps), norm, interleaved)
        return qk_norm_rope_fwd(q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, positions, inv_freq = ctx.saved_tensors
        r = qk_norm_rope_bwd(q, k, q_weight, k_weight, positions, inv_freq, _gradient(dq_out),
                             None if k is None else _gradient(dk_out), *ctx.args)
        return r["dq"], r["dk"], r["dq_weight"], r["dk_weight"], None, None, None, None, None


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, positions=None, inv_freq=None, eps: float = 1e-6,
                 norm: str = "rms", interleaved: bool = False):
    """qk_norm_rope_fwd with autograd support; the gradients reach q, k, q_weight and k_weight."""
    return QkNormRope.apply(q, k, q_weight, k_weight, positions, inv_freq, eps, norm, interleaved)
