"""ctypes binding of the norms before and after a block of libssd_bwd.so (include/block_norm.h).

Argument marshalling only, as in ``ssd``; every arithmetic step runs in the
library's kernels, and the calls raise if the library is missing or returns
an error.

``add_norm`` stands before a block (the residual's sum and the norm of it),
``gated_norm`` after one (the norm with the gate, and the residual's sum where
one is given).  ``*_fwd`` and ``*_bwd`` are the entry points that they pair as
autograd functions.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from state_space_model_mamba_amd import ssd
from state_space_model_mamba_amd.delta import _gradient, _on, _stream

F32 = torch.float32

NORMS = {"rms": 0, "layer": 1}
GATES = {"silu": 0, "sigmoid": 1}
EXPORTED = ("add_norm_fwd", "add_norm_bwd", "gated_norm_fwd", "gated_norm_bwd", "block_norm_bwd_workspace_size")


class BlockNormShape(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("batch", "seqlen", "width", "groups", "x_batch_stride", "x_row_stride",
                                               "z_batch_stride", "z_row_stride")] +
                [(n, ctypes.c_int32) for n in ("norm", "gate", "norm_before_gate", "io_dtype", "residual_dtype",
                                               "reserved")] +
                [("eps", ctypes.c_float), ("alpha", ctypes.c_float)])


_lib = None


def load_library():
    """The shared library with the block norm entry points' argument types set (raises if it is not built)."""
    global _lib
    if _lib is None:
        lib = ssd.load_library()
        vp, sp, n = ctypes.c_void_p, ctypes.POINTER(BlockNormShape), ctypes.c_size_t
        for name, pointers in (("add_norm_fwd", 8), ("gated_norm_fwd", 8)):
            f = getattr(lib, name)
            f.restype = ctypes.c_int
            f.argtypes = [sp] + [vp] * pointers
        lib.block_norm_bwd_workspace_size.restype = ctypes.c_int
        lib.block_norm_bwd_workspace_size.argtypes = [sp, ctypes.POINTER(n)]
        for name, pointers in (("add_norm_bwd", 12), ("gated_norm_bwd", 12)):
            f = getattr(lib, name)
            f.restype = ctypes.c_int
            f.argtypes = [sp] + [vp] * pointers + [n, vp]
        _lib = lib
    return _lib


def make_shape(batch, seqlen, width, groups=1, norm="rms", gate="silu", norm_before_gate=False,
               io_dtype=ssd.SSD_IO_BF16, residual_dtype=None, eps=1e-6, alpha=1.0, strides=(0, 0, 0, 0)) -> BlockNormShape:
    norm = NORMS[norm] if isinstance(norm, str) else int(norm)
    gate = GATES[gate] if isinstance(gate, str) else int(gate)
    return BlockNormShape(batch, seqlen, width, groups, *strides, norm, gate, int(norm_before_gate), io_dtype,
                          io_dtype if residual_dtype is None else residual_dtype, 0, eps, alpha)


def workspace_size(shape: BlockNormShape) -> int:
    """Bytes of workspace that add_norm_bwd or gated_norm_bwd needs."""
    n = ctypes.c_size_t(0)
    rc = load_library().block_norm_bwd_workspace_size(ctypes.byref(shape), ctypes.byref(n))
    if rc:
        raise ssd.SsdError(rc, "block_norm_bwd_workspace_size")
    return n.value


@functools.lru_cache(maxsize=256)
def _sized(*sizes) -> tuple[BlockNormShape, int]:
    """make_shape and its workspace size, kept per sizes (callers read them only)."""
    shape = make_shape(*sizes)
    return shape, workspace_size(shape)


def row_strides(t, name):
    """(batch, row) strides of a (batch, rows, width) tensor whose last axis is contiguous; 0, 0: contiguous."""
    if t.is_contiguous():
        return 0, 0
    b, L, w = t.shape
    sb, sl, sw = t.stride()
    if sw != 1 and w > 1:
        raise ValueError(f"{name} must be contiguous in its last axis")
    if L == 1:
        sl = w
    if b == 1:
        sb = L * sl or w   # one row for all: any step that is not 0 (0, 0 says contiguous)
    if sb == 0 and sl == 0:
        raise ValueError(f"{name} may be broadcast over batch or rows, not over both")
    return sb, sl


def _strided(t, name, dtype, shape, device):
    if t is None:
        return 0, 0
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return row_strides(t, name)


def _check(t, name, dtype, shape, device):
    """ssd._check, its messages formed only where something is wrong."""
    if t is not None and (t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous()):
        ssd._check(t, name, dtype, shape, device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name, function, device, *args):
    """function(*args, stream) with the tensors' device current (the library launches on the current device)."""
    if torch._C._cuda_getDevice() == device.index:
        rc = function(*args, _stream(device))
    else:
        with _on(device):
            rc = function(*args, _stream(device))
    if rc:
        raise ssd.SsdError(rc, name)


def _like(t, dtype=None):
    """An uninitialised contiguous tensor of t's shape."""
    if t.is_contiguous():
        return torch.empty_like(t) if dtype is None or dtype == t.dtype else torch.empty_like(t, dtype=dtype)
    return t.new_empty(t.shape, dtype=dtype)


def _io(dtype):
    return ssd.SSD_IO_BF16 if dtype == torch.bfloat16 else ssd.SSD_IO_F32


def _common(what, x, z, weight, bias, residual, residual_dtype, scale, groups, eps, norm, gate, norm_before_gate):
    """(shape, workspace bytes, scale as a tensor or None, dtype of the residual)"""
    dev, io = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError(f"{what} runs on a HIP device; got tensors on {dev}")
    if io != torch.bfloat16 and io != F32:
        raise ValueError(f"unsupported io dtype {io}")
    if norm not in NORMS:
        raise ValueError(f"norm is one of {sorted(NORMS)}; got {norm!r}")
    if gate not in GATES:
        raise ValueError(f"gate is one of {sorted(GATES)}; got {gate!r}")
    size = x.shape
    if len(size) != 3:
        raise ValueError("x is (batch, seqlen, width)")
    b, L, D = size
    strides = (*row_strides(x, "x"), *_strided(z, "z", io, size, dev))
    if residual is not None:
        if residual_dtype is not None and residual_dtype != residual.dtype:
            raise ValueError(f"residual has dtype {residual.dtype}, residual_dtype is {residual_dtype}")
        residual_dtype = residual.dtype
    elif residual_dtype is None:
        residual_dtype = io
    if residual_dtype != io and residual_dtype != F32:
        raise ValueError(f"the residual's dtype is {io} or float32; got {residual_dtype}")
    vector = (D,)
    _check(residual, "residual", residual_dtype, size, dev)
    _check(weight, "weight", F32, vector, dev)
    _check(bias, "bias", F32, vector, dev)
    alpha = 1.0
    if isinstance(scale, torch.Tensor):
        _check(scale, "scale", F32, vector, dev)
    elif scale is not None:
        alpha, scale = float(scale), None
    shape, nbytes = _sized(b, L, D, int(groups), norm, gate, bool(norm_before_gate), _io(io), _io(residual_dtype),
                           float(eps), alpha, strides)
    return shape, nbytes, scale, residual_dtype


def _workspace(workspace, nbytes, dev):
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev), nbytes
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


def _sum(x, wanted):
    return x.new_empty((x.shape[2],), dtype=F32) if wanted else None


def add_norm_fwd(x, residual=None, weight=None, bias=None, scale=1.0, eps: float = 1e-6, norm: str = "rms",
                 residual_dtype=None):
    """(y, r) with r = residual + scale * x and y = norm(r) * weight + bias.

    x: (b, L, D) bf16 or fp32 (a slice of wider rows is taken as it is); residual: (b, L, D) of x's dtype or fp32, or
    None (r then has ``residual_dtype``, x's by default); weight, bias: (D) fp32 or None; scale: a number, or (D)
    fp32; norm: "rms" (r / sqrt(mean r^2 + eps)) or "layer" (its mean taken off first).  y has x's dtype and is formed
    from the sum before it is rounded to r's.
    """
    shape, _, scale, rdtype = _common("add_norm", x, None, weight, bias, residual, residual_dtype, scale, 1, eps, norm,
                                      "silu", False)
    y = _like(x)
    r = _like(x, rdtype)
    _call("add_norm_fwd", load_library().add_norm_fwd, x.device, shape, x.data_ptr(), _ptr(residual), _ptr(weight),
          _ptr(bias), _ptr(scale), y.data_ptr(), r.data_ptr())
    return y, r


def add_norm_bwd(x, residual, weight, scale, dy, dr, eps: float = 1e-6, norm: str = "rms", residual_dtype=None,
                 want_dresidual: Optional[bool] = None, want_dweight: Optional[bool] = None, want_dbias: bool = False,
                 want_dscale: Optional[bool] = None, workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of sum(dy * y) + sum(dr * r) of add_norm_fwd from its inputs; dy or dr may be None (zeros).

    A dict with dx (like x, contiguous), dresidual (in the residual's dtype; the same tensor as dx where they hold the
    same values), dweight, dbias and dscale ((D) fp32; beside a number the scale counts as a vector of ones).  By
    default those of the inputs that are given (dbias: on demand); the others are None.
    """
    shape, nbytes, scale, rdtype = _common("add_norm", x, None, weight, None, residual, residual_dtype, scale, 1, eps,
                                           norm, "silu", False)
    dev, size = x.device, x.shape
    if dy is None and dr is None:
        raise ValueError("add_norm_bwd needs dy or dr")
    _check(dy, "dy", x.dtype, size, dev)
    _check(dr, "dr", rdtype, size, dev)
    workspace, nbytes = _workspace(workspace, nbytes, dev)
    want_dresidual = residual is not None if want_dresidual is None else want_dresidual
    same = scale is None and shape.alpha == 1.0 and rdtype == x.dtype
    out = {"dx": _like(x),
           "dresidual": _like(x, rdtype) if want_dresidual and not same else None,
           "dweight": _sum(x, weight is not None if want_dweight is None else want_dweight),
           "dbias": _sum(x, want_dbias),
           "dscale": _sum(x, scale is not None if want_dscale is None else want_dscale)}
    _call("add_norm_bwd", load_library().add_norm_bwd, dev, shape, x.data_ptr(), _ptr(residual), _ptr(weight),
          _ptr(scale), _ptr(dy), _ptr(dr), out["dx"].data_ptr(), _ptr(out["dresidual"]), _ptr(out["dweight"]),
          _ptr(out["dbias"]), _ptr(out["dscale"]), workspace.data_ptr(), nbytes)
    if want_dresidual and same:
        out["dresidual"] = out["dx"]
    return out


class AddNorm(torch.autograd.Function):
    """add_norm_fwd paired with add_norm_bwd (deterministic); only the inputs are kept between the two."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, scale, eps, norm, residual_dtype):
        ctx.set_materialize_grads(False)
        y, r = add_norm_fwd(x, residual, weight, bias, scale, eps, norm, residual_dtype)
        tensor = isinstance(scale, torch.Tensor)
        ctx.save_for_backward(x, residual, weight, scale if tensor else None)
        ctx.alpha = None if tensor else scale
        ctx.args = (float(eps), norm, r.dtype)
        return y, r

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr):
        if dy is None and dr is None:
            return (None,) * 8
        x, residual, weight, scale = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = add_norm_bwd(x, residual, weight, ctx.alpha if scale is None else scale,
                         None if dy is None else _gradient(dy), None if dr is None else _gradient(dr), *ctx.args,
                         want_dresidual=need[1], want_dweight=need[2], want_dbias=need[3], want_dscale=need[4])
        return (g["dx"] if need[0] else None), g["dresidual"], g["dweight"], g["dbias"], g["dscale"], None, None, None


def add_norm(x, residual=None, weight=None, bias=None, scale=1.0, eps: float = 1e-6, norm: str = "rms",
             residual_dtype=None):
    """add_norm_fwd with autograd support; gradients reach x, residual, weight, bias and a scale that is a tensor,
    from y and from r."""
    return AddNorm.apply(x, residual, weight, bias, scale, eps, norm, residual_dtype)


def gated_norm_fwd(x, z=None, weight=None, bias=None, residual=None, scale=1.0, groups: int = 1, eps: float = 1e-6,
                   norm: str = "rms", gate: str = "silu", norm_before_gate: bool = False):
    """scale * n, or residual + scale * n, with n = norm(x * act(z)) * weight + bias, or with ``norm_before_gate``
    (norm(x) * weight + bias) * act(z).

    x, z: (b, L, D) in bf16 or fp32 (slices of wider rows are taken as they are; z may be None, and act is then 1);
    the norm is taken over each of ``groups`` runs of D / groups channels; gate: "silu" or "sigmoid"; weight, bias,
    scale and norm as for add_norm_fwd; residual: (b, L, D) of x's dtype or fp32, or None.  The result has the
    residual's dtype (x's without one).
    """
    shape, _, scale, rdtype = _common("gated_norm", x, z, weight, bias, residual, None, scale, groups, eps, norm, gate,
                                      norm_before_gate)
    out = _like(x, rdtype)
    _call("gated_norm_fwd", load_library().gated_norm_fwd, x.device, shape, x.data_ptr(), _ptr(z), _ptr(weight),
          _ptr(bias), _ptr(residual), _ptr(scale), out.data_ptr())
    return out


def gated_norm_bwd(x, z, weight, bias, scale, dout, groups: int = 1, eps: float = 1e-6, norm: str = "rms",
                   gate: str = "silu", norm_before_gate: bool = False, want_dweight: Optional[bool] = None,
                   want_dbias: Optional[bool] = None, want_dscale: Optional[bool] = None,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of sum(dout * out) of gated_norm_fwd from its inputs (that of the residual is dout, whose dtype is
    the residual's).

    A dict with dx, dz (like x, contiguous; dz None without z), dweight, dbias and dscale ((D) fp32; by default those
    of the inputs that are given, the others are None).
    """
    shape, nbytes, scale, rdtype = _common("gated_norm", x, z, weight, bias, None, dout.dtype, scale, groups, eps, norm,
                                           gate, norm_before_gate)
    dev = x.device
    _check(dout, "dout", rdtype, x.shape, dev)
    workspace, nbytes = _workspace(workspace, nbytes, dev)
    out = {"dx": _like(x),
           "dz": None if z is None else _like(x),
           "dweight": _sum(x, weight is not None if want_dweight is None else want_dweight),
           "dbias": _sum(x, bias is not None if want_dbias is None else want_dbias),
           "dscale": _sum(x, scale is not None if want_dscale is None else want_dscale)}
    _call("gated_norm_bwd", load_library().gated_norm_bwd, dev, shape, x.data_ptr(), _ptr(z), _ptr(weight), _ptr(bias),
          _ptr(scale), dout.data_ptr(), out["dx"].data_ptr(), _ptr(out["dz"]), _ptr(out["dweight"]),
          _ptr(out["dbias"]), _ptr(out["dscale"]), workspace.data_ptr(), nbytes)
    return out


class GatedNorm(torch.autograd.Function):
    """gated_norm_fwd paired with gated_norm_bwd (deterministic); only the inputs are kept between the two."""

    @staticmethod
    def forward(ctx, x, z, weight, bias, residual, scale, groups, eps, norm, gate, norm_before_gate):
        ctx.set_materialize_grads(False)
        tensor = isinstance(scale, torch.Tensor)
        ctx.save_for_backward(x, z, weight, bias, scale if tensor else None)
        ctx.alpha = None if tensor else scale
        ctx.args = (int(groups), float(eps), norm, gate, bool(norm_before_gate))
        return gated_norm_fwd(x, z, weight, bias, residual, scale, groups, eps, norm, gate, norm_before_gate)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        if dout is None:
            return (None,) * 11
        x, z, weight, bias, scale = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = gated_norm_bwd(x, z, weight, bias, ctx.alpha if scale is None else scale, _gradient(dout), *ctx.args,
                           want_dweight=need[2], want_dbias=need[3], want_dscale=need[5])
        return ((g["dx"] if need[0] else None), (g["dz"] if need[1] else None), g["dweight"], g["dbias"],
                (dout if need[4] else None), g["dscale"], None, None, None, None, None)


def gated_norm(x, z=None, weight=None, bias=None, residual=None, scale=1.0, groups: int = 1, eps: float = 1e-6,
               norm: str = "rms", gate: str = "silu", norm_before_gate: bool = False):
    """gated_norm_fwd with autograd support; gradients reach x, z, weight, bias, residual and a scale that is a
    tensor."""
    return GatedNorm.apply(x, z, weight, bias, residual, scale, groups, eps, norm, gate, norm_before_gate)
