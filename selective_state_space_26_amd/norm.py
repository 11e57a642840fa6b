"""Python binding of the norms around a block (argument marshalling only: the HIP kernels of
libmsel.so do the work).

Layouts, as in include/msel.h:

    x, out, dout, dx            : [..., dim]  float32 or bfloat16, contiguous
    residual, s, dresidual, ... : [..., dim]  the same dtype, or float32 beside bfloat16
    weight, dweight             : [dim]       float32

and for the gated norm

    x, z, dx, dz                : [batch, dim, seqlen] ("bdl") or [batch, seqlen, dim] ("bld")
    out, dout                   : the same, or "bld" for x in "bdl"
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .scan import _dtype_code, _int32, _need, _stream, _workspace

_LAYOUTS = {"bdl": 0, "bld": 1}


# the current stream's handle without a Stream object around it (2 us less per call), where this
# build of PyTorch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(dev):
    """The current stream of a GPU, as the library takes it."""
    return _stream(dev) if _raw_stream is None else _raw_stream(dev.index)


def _at(t):
    return None if t is None else t.data_ptr()


def _rows(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() < 1 or t.numel() == 0:
        raise ValueError(f"{name} must be a non-empty [..., dim] tensor")
    if t.device.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    dim = _int32(t.shape[-1], "dim")
    return t.shape, dim, t.numel() // dim


def msel_norm_fwd(x, weight=None, residual=None, scale=1.0, eps=1e-5, residual_dtype=None,
                  out=None, residual_out=None):
    """RMS norm before a block: s = residual + scale * x (scale * x without a residual),
    out = s / sqrt(mean(s^2) + eps) * weight over the last axis.

    Returns (out, residual_out): residual_out holds s in the residual's dtype, in
    `residual_dtype` when there is no residual, and is None when neither is given.  A given
    residual_out may be `residual` itself, which is then updated in place."""
    shape, dim, rows = _rows(x, "x")
    dev, dt = x.device, x.dtype
    code = _dtype_code(dt)
    _need(x, "x", shape, dt, dev)
    _need(weight, "weight", (dim,), torch.float32, dev)
    rdt = residual_dtype or (residual if residual is not None else
                             residual_out if residual_out is not None else x).dtype
    rcode = _dtype_code(rdt)
    _need(residual, "residual", shape, rdt, dev)
    out = torch.empty_like(x) if out is None else _need(out, "out", shape, dt, dev)
    if residual_out is not None:
        _need(residual_out, "residual_out", shape, rdt, dev)
    elif residual is not None:
        residual_out = torch.empty_like(residual)
    elif residual_dtype is not None:
        residual_out = torch.empty(shape, device=dev, dtype=rdt)
    a = _lib.NormArgs(_lib.ABI_VERSION, dim, rows, code, rcode, scale, eps, x.data_ptr(),
                      _at(residual), _at(weight), out.data_ptr(), _at(residual_out))
    _lib.check("msel_norm_fwd", _lib.load().msel_norm_fwd(ctypes.byref(a), _handle(dev)))
    return out, residual_out


def msel_norm_bwd(s, weight, dout, dresidual_out=None, scale=1.0, eps=1e-5, want_dx=True,
                  want_dresidual=True, want_dweight=True, dresidual=None, workspace=None):
    """Gradients of sum(dout * out) + sum(dresidual_out * residual_out) for msel_norm_fwd, whose
    residual_out is `s` (scale * x when the call had no residual).  A given dresidual may be
    dresidual_out itself.  Returns {"dx", "dresidual", "dweight"} (absent ones are None)."""
    shape, dim, rows = _rows(s, "s")
    dev, rdt = s.device, s.dtype
    if not isinstance(dout, torch.Tensor):
        raise TypeError("dout must be a torch.Tensor")
    dt = dout.dtype
    code, rcode = _dtype_code(dt), _dtype_code(rdt)
    _need(s, "s", shape, rdt, dev)
    _need(weight, "weight", (dim,), torch.float32, dev)
    _need(dout, "dout", shape, dt, dev)
    _need(dresidual_out, "dresidual_out", shape, rdt, dev)
    _need(dresidual, "dresidual", shape, rdt, dev)
    dx = torch.empty_like(dout) if want_dx else None
    if dresidual is None and want_dresidual:
        dresidual = torch.empty_like(s)
    dw = torch.empty((dim,), device=dev, dtype=torch.float32) if want_dweight else None
    a = _lib.NormArgs(_lib.ABI_VERSION, dim, rows, code, rcode, scale, eps, None, None,
                      _at(weight), None, None)
    g = _lib.NormGrads(s.data_ptr(), dout.data_ptr(), _at(dresidual_out), _at(dx),
                       _at(dresidual), _at(dw))
    lib = _lib.load()
    need = lib.msel_norm_bwd_workspace_bytes(ctypes.byref(a)) if want_dweight else 0
    workspace, size = _workspace(workspace, need, dev)
    _lib.check("msel_norm_bwd", lib.msel_norm_bwd(ctypes.byref(a), ctypes.byref(g),
                                                  _at(workspace), size, _handle(dev)))
    return {"dx": dx, "dresidual": dresidual, "dweight": dw}


def _gated_args(x, z, weight, eps, groups, gate_first, layout, out_layout):
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [batch, dim, seqlen] or [batch, seqlen, dim] tensor")
    if layout not in _LAYOUTS or out_layout not in _LAYOUTS:
        raise ValueError(f"layouts are {sorted(_LAYOUTS)}, got {layout!r} and {out_layout!r}")
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    code = _dtype_code(dt)
    bsz = x.shape[0]
    dim, L = (x.shape[1], x.shape[2]) if layout == "bdl" else (x.shape[2], x.shape[1])
    _need(x, "x", x.shape, dt, dev)
    if z is None:
        raise TypeError("z must be a torch.Tensor")
    _need(z, "z", x.shape, dt, dev)
    _need(weight, "weight", (dim,), torch.float32, dev)
    a = _lib.GatedNormArgs(_lib.ABI_VERSION, _int32(bsz, "batch"), _int32(dim, "dim"),
                           _int32(L, "seqlen"), _int32(groups, "groups"), code,
                           _LAYOUTS[layout], _LAYOUTS[out_layout], 1 if gate_first else 0, eps,
                           x.data_ptr(), z.data_ptr(), _at(weight), None)
    return a, ((bsz, dim, L) if out_layout == "bdl" else (bsz, L, dim))


def msel_gated_norm_fwd(x, z, weight=None, eps=1e-5, groups=1, gate_first=True, layout="bdl",
                        out_layout=None, out=None):
    """RMS norm of the scan's output over its channels (over each of `groups` equal parts of
    them), fused with the gate: norm(x * silu(z)) * weight when gate_first, else
    norm(x) * weight * silu(z).  x is the scan's output without its own gate (z=None there).
    out_layout (default: layout) may be "bld" for "bdl" inputs.  Returns out."""
    a, shape = _gated_args(x, z, weight, eps, groups, gate_first, layout, out_layout or layout)
    dev = x.device
    out = (x.new_empty(shape) if out is None
           else _need(out, "out", shape, x.dtype, dev))
    a.out = out.data_ptr()
    _lib.check("msel_gated_norm_fwd",
               _lib.load().msel_gated_norm_fwd(ctypes.byref(a), _handle(dev)))
    return out


def msel_gated_norm_bwd(x, z, weight, dout, eps=1e-5, groups=1, gate_first=True, layout="bdl",
                        out_layout=None, want_dweight=True, workspace=None):
    """Gradients of sum(dout * out) for msel_gated_norm_fwd's out, recomputing the gate and the
    norm.  Returns {"dx", "dz", "dweight"} (dweight is None unless wanted)."""
    a, shape = _gated_args(x, z, weight, eps, groups, gate_first, layout, out_layout or layout)
    dev = x.device
    if dout is None:
        raise TypeError("dout must be a torch.Tensor")
    _need(dout, "dout", shape, x.dtype, dev)
    dx, dz = torch.empty_like(x), torch.empty_like(x)
    dw = torch.empty((a.dim,), device=dev, dtype=torch.float32) if want_dweight else None
    g = _lib.GatedNormGrads(dout.data_ptr(), dx.data_ptr(), dz.data_ptr(), _at(dw))
    lib = _lib.load()
    need = lib.msel_gated_norm_bwd_workspace_bytes(ctypes.byref(a)) if want_dweight else 0
    workspace, size = _workspace(workspace, need, dev)
    _lib.check("msel_gated_norm_bwd",
               lib.msel_gated_norm_bwd(ctypes.byref(a), ctypes.byref(g), _at(workspace), size,
                                       _handle(dev)))
    return {"dx": dx, "dz": dz, "dweight": dw}
