"""Python binding of the embedding lookup and its gradient (argument marshalling only).

Layouts, as in include/msel.h:

    ids           : [...]        int64 or int32, contiguous
    weight        : [vocab, dim] float32 or bfloat16
    out, dout     : [..., dim]   float32 or bfloat16
    dweight, base : [vocab, dim] float32
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .norm import _at, _handle
from .scan import _dtype_code, _int32, _need, _workspace


def _embed_args(ids, vocab, dim, scale, padding_idx, code, wcode):
    if not isinstance(ids, torch.Tensor) or ids.numel() == 0:
        raise ValueError("ids must be a non-empty tensor")
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"ids must be int64 or int32, got {ids.dtype}")
    dev = ids.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    _need(ids, "ids", ids.shape, ids.dtype, dev)
    if padding_idx is None or not 0 <= padding_idx < vocab:
        padding_idx = -1  # none: other ids give no gradient anyway
    return _lib.EmbedArgs(_lib.ABI_VERSION, _int32(vocab, "vocab"), _int32(dim, "dim"),
                          1 if ids.dtype == torch.int64 else 0, ids.numel(), padding_idx, code,
                          wcode, scale, 0, ids.data_ptr(), None, None)


def msel_embed_fwd(ids, weight, scale=1.0, dtype=None, out=None):
    """out[..., :] = scale * weight[ids], in `dtype` (default: the table's).  An id outside the
    table gives a row of zeros."""
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [vocab, dim] tensor")
    vocab, dim = weight.shape
    dt = dtype or (weight if out is None else out).dtype
    a = _embed_args(ids, vocab, dim, scale, None, _dtype_code(dt), _dtype_code(weight.dtype))
    dev = ids.device
    _need(weight, "weight", (vocab, dim), weight.dtype, dev)
    shape = (*ids.shape, dim)
    out = (torch.empty(shape, device=dev, dtype=dt) if out is None
           else _need(out, "out", shape, dt, dev))
    a.weight, a.out = weight.data_ptr(), out.data_ptr()
    _lib.check("msel_embed_fwd", _lib.load().msel_embed_fwd(ctypes.byref(a), _handle(dev)))
    return out


def msel_embed_bwd(ids, dout, vocab, scale=1.0, base=None, padding_idx=None, dweight=None,
                   workspace=None):
    """dweight[v] = base[v] + scale * (sum of dout over the tokens with ids == v), fp32
    [vocab, dim]; base None means 0, and a given dweight may be `base` itself (the gradient is
    then added to in place).  Ids outside [0, vocab) and padding_idx give no gradient.  The
    tokens are sorted and added in a fixed order: deterministic."""
    if not isinstance(dout, torch.Tensor) or dout.dim() < 1:
        raise ValueError("dout must be an [..., dim] tensor")
    dim = dout.shape[-1]
    a = _embed_args(ids, vocab, dim, scale, padding_idx, _dtype_code(dout.dtype), 0)
    dev = ids.device
    _need(dout, "dout", (*ids.shape, dim), dout.dtype, dev)
    _need(base, "base", (vocab, dim), torch.float32, dev)
    dweight = (torch.empty((vocab, dim), device=dev, dtype=torch.float32) if dweight is None
               else _need(dweight, "dweight", (vocab, dim), torch.float32, dev))
    g = _lib.EmbedGrads(dout.data_ptr(), _at(base), dweight.data_ptr())
    lib = _lib.load()
    workspace, size = _workspace(workspace, lib.msel_embed_bwd_workspace_bytes(ctypes.byref(a)),
                                 dev)
    _lib.check("msel_embed_bwd", lib.msel_embed_bwd(ctypes.byref(a), ctypes.byref(g),
                                                    _at(workspace), size, _handle(dev)))
    return dweight
