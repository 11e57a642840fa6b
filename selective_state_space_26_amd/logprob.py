"""Python binding of the log probabilities of tokens (argument marshalling only: the HIP kernels of
libmsel.so do the work).

Layouts, as in include/msel.h:

    logits, dlogits                      : [..., vocab]  float32 or bfloat16; rows may be strided
                                           alike (the first columns of a padded vocabulary)
    ids                                  : [...]         int64 or int32
    logprob, lse, entropy and gradients  : [...]         float32
    top_ids, top_logprobs                : [..., top]    int64, float32
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from .lru import _call
from .norm import _at
from .scan import _dtype_code, _int32, _need, _workspace


def _strided(t, name):
    """(rows, elements from a row to the next) of [..., vocab] with consecutive columns."""
    vocab = t.shape[-1]
    rows = t.numel() // vocab
    if vocab > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have consecutive columns")
    step, n = None, 1  # the rows' stride, and the rows inside the axes seen so far
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if step is None:
            step = stride
        if stride != step * n:
            raise ValueError(f"the rows of {name} must be strided alike")
        n *= size
    return rows, vocab if step is None else step


@functools.lru_cache(maxsize=1024)
def _need_bytes(rows, vocab, top, code):
    """Bytes of workspace the forward needs for these sizes."""
    a = _lib.LogprobArgs(_lib.ABI_VERSION, vocab, rows, vocab, code, 0, top, 1.0)
    return _lib.load().msel_logprob_fwd_workspace_bytes(ctypes.byref(a))


def _args(logits, ids, scale):
    if not isinstance(logits, torch.Tensor) or logits.dim() < 1 or logits.numel() == 0:
        raise ValueError("logits must be a non-empty [..., vocab] tensor")
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    code = _dtype_code(logits.dtype)
    vocab = _int32(logits.shape[-1], "vocab")
    rows, stride = _strided(logits, "logits")
    if ids is not None:
        if not isinstance(ids, torch.Tensor):
            raise TypeError("ids must be a torch.Tensor")
        if ids.dtype not in (torch.int64, torch.int32):
            raise TypeError(f"ids must be int64 or int32, got {ids.dtype}")
        _need(ids, "ids", logits.shape[:-1], ids.dtype, dev)
    a = _lib.LogprobArgs()
    a.abi_version, a.vocab, a.rows, a.stride = _lib.ABI_VERSION, vocab, rows, stride
    a.dtype, a.scale, a.logits = code, scale, logits.data_ptr()
    a.ids_64bit = 1 if ids is None or ids.dtype == torch.int64 else 0
    a.ids = _at(ids)
    return a


def msel_logprob_fwd(logits, ids=None, scale=1.0, top=0, want_lse=True, want_entropy=False,
                     workspace=None):
    """Log probabilities under softmax(scale * logits) over the last axis: of the token `ids` of
    each row (0 for an id outside the vocabulary), and of the `top` (up to 64) likeliest tokens,
    in falling order and by the lowest id where logits are equal.

    Returns {"logprob", "lse", "entropy", "top_ids", "top_logprobs"} (absent ones are None)."""
    a = _args(logits, ids, scale)
    a.top = _int32(top, "top")
    dev, shape = logits.device, logits.shape[:-1]

    def rows(*more, dtype=torch.float32):
        size = (*shape, *more)  # one by one: 0.8 us less than as a torch.Size
        if not size:
            return torch.empty((), device=dev, dtype=dtype)
        return torch.empty(*size, device=dev, dtype=dtype)
    logprob = rows() if ids is not None else None
    lse = rows() if want_lse else None
    entropy = rows() if want_entropy else None
    top_ids = rows(top, dtype=torch.int64) if top > 0 else None
    top_logprobs = rows(top) if top > 0 else None
    a.logprob, a.lse, a.entropy = _at(logprob), _at(lse), _at(entropy)
    a.top_ids, a.top_logprobs = _at(top_ids), _at(top_logprobs)
    need = _need_bytes(a.rows, a.vocab, a.top, a.dtype)
    workspace, size = _workspace(workspace, need, dev)
    _call("msel_logprob_fwd", dev, ctypes.byref(a), _at(workspace), size)
    return {"logprob": logprob, "lse": lse, "entropy": entropy, "top_ids": top_ids,
            "top_logprobs": top_logprobs}


def msel_logprob_bwd(logits, ids, lse, dlogprob=None, dlse=None, dentropy=None, entropy=None,
                     scale=1.0, dlogits=None):
    """Gradient of sum(dlogprob * logprob) + sum(dlse * lse) + sum(dentropy * entropy) for
    msel_logprob_fwd, given its lse (and its entropy where dentropy is given).  Returns dlogits,
    contiguous unless given; a given one may be `logits` itself, which is then overwritten."""
    a = _args(logits, ids, scale)
    dev, shape = logits.device, logits.shape[:-1]
    if lse is None:
        raise TypeError("lse must be a torch.Tensor")
    for name, t in (("lse", lse), ("entropy", entropy), ("dlogprob", dlogprob), ("dlse", dlse),
                    ("dentropy", dentropy)):
        _need(t, name, shape, torch.float32, dev)
    a.lse, a.entropy = lse.data_ptr(), _at(entropy)
    if dlogits is None:
        dlogits = torch.empty(*logits.shape, device=dev, dtype=logits.dtype)
        dstride = a.vocab
    else:
        if not isinstance(dlogits, torch.Tensor):
            raise TypeError("dlogits must be a torch.Tensor")
        if dlogits.device != dev or dlogits.dtype != logits.dtype:
            raise ValueError("dlogits must have the logits' device and dtype")
        if dlogits.shape != logits.shape:
            raise ValueError(f"dlogits has shape {tuple(dlogits.shape)}, expected "
                             f"{tuple(logits.shape)}")
        dstride = _strided(dlogits, "dlogits")[1]
    g = _lib.LogprobGrads(_at(dlogprob), _at(dlse), _at(dentropy), dlogits.data_ptr(), dstride)
    _call("msel_logprob_bwd", dev, ctypes.byref(a), ctypes.byref(g))
    return dlogits
