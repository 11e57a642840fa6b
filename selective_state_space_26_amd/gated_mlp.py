"""Python binding of the gated feed-forward block (argument marshalling only: the HIP kernels of
libmsel.so do the work).

Layouts, as in include/msel.h, all float32 or all bfloat16, contiguous:

    x, dx                    : [..., dim]
    w_gate, w_up, gradients  : [hidden, dim]
    out, dout                : [..., hidden]
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from .lru import _call
from .norm import _at, _rows
from .scan import _dtype_code, _int32, _need, _workspace

_ACTIVATIONS = {"silu": 0, "gelu": 1}


@functools.lru_cache(maxsize=1024)
def _need_bytes(fn, dim, hidden, code, tokens):
    """Bytes of workspace for these sizes."""
    a = _lib.GatedMlpArgs(_lib.ABI_VERSION, dim, hidden, code, tokens, 0, 0)
    return getattr(_lib.load(), fn)(ctypes.byref(a))


def _args(x, w_gate, w_up, activation):
    shape, dim, tokens = _rows(x, "x")
    if not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2:
        raise ValueError("w_gate must be a [hidden, dim] tensor")
    if w_up is None:
        raise TypeError("w_up must be a torch.Tensor")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation is one of {sorted(_ACTIVATIONS)}, got {activation!r}")
    dev, dt = x.device, x.dtype
    code = _dtype_code(dt)
    hidden = _int32(w_gate.shape[0], "hidden")
    _need(x, "x", shape, dt, dev)
    _need(w_gate, "w_gate", (hidden, dim), dt, dev)
    _need(w_up, "w_up", (hidden, dim), dt, dev)
    a = _lib.GatedMlpArgs(_lib.ABI_VERSION, dim, hidden, code, tokens, _ACTIVATIONS[activation], 0,
                          x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), None)
    return a, shape[:-1] + (hidden,)


def msel_gated_mlp_fwd(x, w_gate, w_up, activation="silu", out=None, workspace=None):
    """act(x @ w_gate.T) * (x @ w_up.T) in one kernel; activation "silu" or "gelu" (its tanh form).
    Returns out."""
    a, shape = _args(x, w_gate, w_up, activation)
    dev = x.device
    out = x.new_empty(shape) if out is None else _need(out, "out", shape, x.dtype, dev)
    a.out = out.data_ptr()
    need = _need_bytes("msel_gated_mlp_fwd_workspace_bytes", a.dim, a.hidden, a.dtype, a.tokens)
    workspace, size = _workspace(workspace, need, dev)
    _call("msel_gated_mlp_fwd", dev, ctypes.byref(a), _at(workspace), size)
    return out


def msel_gated_mlp_bwd(x, w_gate, w_up, dout, activation="silu", want_dx=True,
                       want_dweights=True, workspace=None):
    """Gradients of sum(dout * out) for msel_gated_mlp_fwd, forming both projections again.
    Returns {"dx", "dw_gate", "dw_up"}, in x's dtype (absent ones are None).  In bfloat16 the
    gradients of the projections are rounded once between the products, to one bfloat16 number or,
    up to tokens * min(dim, hidden) = 4096, to two."""
    a, shape = _args(x, w_gate, w_up, activation)
    dev = x.device
    if dout is None:
        raise TypeError("dout must be a torch.Tensor")
    _need(dout, "dout", shape, x.dtype, dev)
    dx = torch.empty_like(x) if want_dx else None
    dwg, dwu = ((torch.empty_like(w_gate), torch.empty_like(w_up)) if want_dweights
                else (None, None))
    g = _lib.GatedMlpGrads(dout.data_ptr(), _at(dx), _at(dwg), _at(dwu))
    need = _need_bytes("msel_gated_mlp_bwd_workspace_bytes", a.dim, a.hidden, a.dtype, a.tokens)
    workspace, size = _workspace(workspace, need, dev)
    _call("msel_gated_mlp_bwd", dev, ctypes.byref(a), ctypes.byref(g), _at(workspace), size)
    return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}
