"""Python binding of the gated linear recurrence (argument marshalling only: the HIP kernels of
libmsel.so do the work).

Layouts, as in include/msel.h:

    x, gate_a, gate_x, out, dout, dx, ...  : [batch, dim, seqlen]           float32 or bfloat16
    lam, dlam                              : [dim]                          float32
    h0, final_state, dfinal_state, dh0     : [batch, dim]                   float32
    chunk_states                           : [batch, dim, num_chunks(seqlen)] float32
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from .norm import _at, _handle
from .scan import _dtype_code, _int32, _need, _workspace, num_chunks


# the current device's index without torch.cuda's checks around it, where this build of PyTorch has it
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, dev, *args):
    """The library's entry point on the current stream of the tensors' device."""
    call = getattr(_lib.load(), fn)
    if dev.index == _current_device():
        code = call(*args, _handle(dev))
    else:
        with torch.cuda.device(dev):
            code = call(*args, _handle(dev))
    _lib.check(fn, code)


@functools.lru_cache(maxsize=1024)
def _need_bytes(fn, bsz, dim, L, code, chunks):
    """Bytes of workspace for these sizes; chunks: the backward is given the chunk states."""
    a = _lib.LruArgs(_lib.ABI_VERSION, bsz, dim, L, code, 0)
    a.chunk_states = 4 if chunks else None
    return getattr(_lib.load(), fn)(ctypes.byref(a))


def _args(x, gate_a, gate_x, lam, h0):
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [batch, dim, seqlen] tensor")
    dev, dt = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    code = _dtype_code(dt)
    shape = bsz, dim, L = x.shape
    for name, t in (("gate_a", gate_a), ("gate_x", gate_x), ("lam", lam)):
        if t is None:
            raise TypeError(f"{name} must be a torch.Tensor")
    _need(x, "x", shape, dt, dev)
    _need(gate_a, "gate_a", shape, dt, dev)
    _need(gate_x, "gate_x", shape, dt, dev)
    _need(lam, "lam", (dim,), torch.float32, dev)
    _need(h0, "h0", (bsz, dim), torch.float32, dev)
    return _lib.LruArgs(_lib.ABI_VERSION, _int32(bsz, "batch"), _int32(dim, "dim"),
                        _int32(L, "seqlen"), code, 0, x.data_ptr(), gate_a.data_ptr(),
                        gate_x.data_ptr(), lam.data_ptr(), _at(h0), None, None, None)


def msel_lru_fwd(x, gate_a, gate_x, lam, h0=None, return_final_state=True,
                 return_chunk_states=False, out=None, final_state=None, chunk_states=None,
                 workspace=None):
    """Gated linear recurrence over time, one state per channel:

        a = exp(lam * sigmoid(gate_a)),  h_t = a h_{t-1} + sqrt(1 - a^2) sigmoid(gate_x) x_t

    with lam <= 0 per channel (a positive one gives NaN).  Returns (out, final_state or None,
    chunk_states or None): out holds every h_t, chunk_states what msel_lru_bwd starts from.  A
    given final_state may be h0 itself, which is then updated in place."""
    a = _args(x, gate_a, gate_x, lam, h0)
    dev, bsz, dim, L = x.device, a.batch, a.dim, a.seqlen
    out = torch.empty_like(x) if out is None else _need(out, "out", x.shape, x.dtype, dev)
    if final_state is not None:
        _need(final_state, "final_state", (bsz, dim), torch.float32, dev)
    elif return_final_state:
        final_state = torch.empty(bsz, dim, device=dev, dtype=torch.float32)
    if chunk_states is not None:
        _need(chunk_states, "chunk_states", (bsz, dim, num_chunks(L)), torch.float32, dev)
    elif return_chunk_states:
        chunk_states = torch.empty(bsz, dim, num_chunks(L), device=dev, dtype=torch.float32)
    a.out, a.final_state, a.chunk_states = out.data_ptr(), _at(final_state), _at(chunk_states)
    need = _need_bytes("msel_lru_fwd_workspace_bytes", bsz, dim, L, a.dtype, False)
    workspace, size = _workspace(workspace, need, dev)
    _call("msel_lru_fwd", dev, ctypes.byref(a), _at(workspace), size)
    return out, final_state, chunk_states


def msel_lru_bwd(x, gate_a, gate_x, lam, dout, h0=None, dfinal_state=None, chunk_states=None,
                 want_dlam=True, want_dh0=False, workspace=None):
    """Gradients of sum(dout * out) + sum(dfinal_state * final_state) for msel_lru_fwd,
    recomputing the states from its chunk_states (or from the start, without them).  Returns
    {"dx", "dgate_a", "dgate_x", "dlam", "dh0"} (absent ones are None)."""
    a = _args(x, gate_a, gate_x, lam, h0)
    dev, (bsz, dim, L) = x.device, x.shape
    if dout is None:
        raise TypeError("dout must be a torch.Tensor")
    _need(dout, "dout", x.shape, x.dtype, dev)
    _need(dfinal_state, "dfinal_state", (bsz, dim), torch.float32, dev)
    _need(chunk_states, "chunk_states", (bsz, dim, num_chunks(L)), torch.float32, dev)
    a.chunk_states = _at(chunk_states)
    dx, dga, dgx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dlam = torch.empty(dim, device=dev, dtype=torch.float32) if want_dlam else None
    dh0 = torch.empty(bsz, dim, device=dev, dtype=torch.float32) if want_dh0 else None
    g = _lib.LruGrads(dout.data_ptr(), _at(dfinal_state), dx.data_ptr(), dga.data_ptr(),
                      dgx.data_ptr(), _at(dlam), _at(dh0))
    need = _need_bytes("msel_lru_bwd_workspace_bytes", bsz, dim, L, a.dtype,
                       chunk_states is not None)
    workspace, size = _workspace(workspace, need, dev)
    _call("msel_lru_bwd", dev, ctypes.byref(a), ctypes.byref(g), _at(workspace), size)
    return {"dx": dx, "dgate_a": dga, "dgate_x": dgx, "dlam": dlam, "dh0": dh0}
