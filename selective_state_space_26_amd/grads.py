"""Python binding of the gradient norm over many tensors and of clipping (argument marshalling
only).  Tensors are contiguous float32 or bfloat16, of any shapes, on one device."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .norm import _at, _handle
from .scan import _dtype_code, _workspace


class GradList:
    """The tensors of one model, checked once and kept as the library's list of them (with
    references to the tensors and their storages, so that the listed memory stays theirs).

    A program whose gradients are the same tensors at every step builds it once.  PyTorch's
    zero_grad() drops the gradients and the next backward makes new ones: the list then still
    names the old ones, and clipping it leaves the new ones as they are.  Such a program calls
    zero_grad(set_to_none=False), which keeps them, or passes the gradients themselves to every
    call (a list of 266 tensors takes 0.3 ms of the host to build).  One that replaces or resizes
    a listed tensor's storage builds a new list; check() finds the tensors it did that to."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.storages = []
        self.device = None
        self.entries = (_lib.TensorEntry * len(self.tensors))()
        for i, t in enumerate(self.tensors):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"tensor {i} must be a torch.Tensor")
            if t.device.type != "cuda":
                raise ValueError("tensors must be on the GPU")
            if self.device is None:
                self.device = t.device
            if t.device != self.device:
                raise ValueError(f"tensor {i} is on {t.device}, expected {self.device}")
            if not t.is_contiguous():
                raise ValueError(f"tensor {i} must be contiguous")
            self.storages.append(t.untyped_storage())
            self.entries[i] = _lib.TensorEntry(t.data_ptr(), t.numel(), _dtype_code(t.dtype), 0)
        if self.device is None:
            raise ValueError("a GradList needs at least one tensor")
        args = _lib.GradArgs(_lib.ABI_VERSION, len(self.tensors), self.entries, None, 0.0, 0.0,
                             None)
        self.workspace_bytes = _lib.load().msel_grad_workspace_bytes(ctypes.byref(args))

    def __len__(self):
        return len(self.tensors)

    def check(self):
        """Raises if a listed tensor's memory, size or dtype is no longer what the list has."""
        for i, (t, e) in enumerate(zip(self.tensors, self.entries)):
            if (t.data_ptr() != (e.data or 0) or t.numel() != e.numel or not t.is_contiguous()
                    or _dtype_code(t.dtype) != e.dtype
                    or t.untyped_storage().nbytes() < t.numel() * t.element_size()):
                raise ValueError(f"tensor {i} has changed since the list was built")


def _as_list(grads):
    return grads if isinstance(grads, GradList) else GradList(grads)


def _call(fn, grads, outs, max_norm, eps, norm, workspace):
    dev = grads.device
    if norm is None:
        norm = torch.empty((), device=dev, dtype=torch.float32)
    elif norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != dev:
        raise ValueError("norm must be one float32 value on the tensors' device")
    a = _lib.GradArgs(_lib.ABI_VERSION, len(grads.tensors), grads.entries,
                      None if outs is None else outs.entries, max_norm, eps, norm.data_ptr())
    workspace, size = _workspace(workspace, grads.workspace_bytes, dev)
    _lib.check(fn, getattr(_lib.load(), fn)(ctypes.byref(a), _at(workspace), size, _handle(dev)))
    return norm


def msel_grad_norm(grads, norm=None, workspace=None):
    """sqrt of the sum of squares over all elements of `grads` (a GradList or tensors), as a
    float32 value on the GPU."""
    return _call("msel_grad_norm", _as_list(grads), None, 0.0, 0.0, norm, workspace)


def msel_grad_clip(grads, max_norm, eps=1e-6, out=None, norm=None, workspace=None):
    """Scales every tensor by min(1, max_norm / (norm + eps)), in place or into `out` (a GradList
    or tensors of the same sizes and dtypes), and returns the norm before scaling as
    msel_grad_norm does.  Nothing is read back: a norm that is not finite is in the result.
    What is written shares no memory with anything else: a tensor listed twice, views that
    overlap or another entry's tensor in `out` are refused."""
    grads = _as_list(grads)
    outs = grads if out is None else _as_list(out)
    if len(outs) != len(grads):
        raise ValueError(f"out has {len(outs)} tensors, expected {len(grads)}")
    if outs.device != grads.device:
        raise ValueError(f"out is on {outs.device}, expected {grads.device}")
    return _call("msel_grad_clip", grads, outs, max_norm, eps, norm, workspace)
