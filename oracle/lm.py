"""fp64 CPU oracle of the operators around the selective scan: the norms before and after a
block, the embedding, the gradient norm and clipping.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code with the HIP library
and imports nothing from the product package.

Everything is float64 and follows the definitions line by line:

* norm before a block:  s = residual + scale x;  out = s (mean s^2 + eps)^(-1/2) w
* gated norm, gate first: v = x silu(z);  out = v (mean v^2 + eps)^(-1/2) w
* gated norm, gate last:  out = x (mean x^2 + eps)^(-1/2) w silu(z)
  (means over each group of channels; here the channels are the last axis)
* embedding: out[t] = scale w[ids[t]], zeros for an id outside the table
* clipping: norm = sqrt(sum g^2), g min(1, max_norm / (norm + eps))

The gradients are the chain rule of these, by hand.  Beside a gradient, its ``*_terms`` is the
same expression with every term replaced by its magnitude: the scale that the rounding errors
of a computation in fewer bits have, also where the terms cancel.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def _rstd(v, eps):
    return (np.mean(v * v, axis=-1, keepdims=True) + eps) ** -0.5


def norm_fwd(x, w=None, residual=None, scale=1.0, eps=1e-5):
    """(out, s)."""
    s = scale * _f64(x)
    if residual is not None:
        s = s + _f64(residual)
    out = s * _rstd(s, eps)
    return (out if w is None else out * _f64(w)), s


def norm_bwd(s, w, dout, dresidual_out=None, scale=1.0, eps=1e-5):
    """dict of dx, dresidual, dweight and their terms for rows [rows, dim]."""
    s, dout = _f64(s), _f64(dout)
    r = _rstd(s, eps)
    g = dout if w is None else dout * _f64(w)
    ds = r * (g - s * r * r * np.mean(g * s, axis=-1, keepdims=True))
    terms = r * (np.abs(g) + np.abs(s) * r * r * np.mean(np.abs(g * s), axis=-1, keepdims=True))
    if dresidual_out is not None:
        ds = ds + _f64(dresidual_out)
        terms = terms + np.abs(_f64(dresidual_out))
    t = dout * s * r
    return dict(dx=scale * ds, dx_terms=abs(scale) * terms, dresidual=ds, dresidual_terms=terms,
                dweight=t.sum(0), dweight_terms=np.abs(t).sum(0))


def _split(a, groups):
    return a.reshape(*a.shape[:-1], groups, a.shape[-1] // groups)


def gated_fwd(x, z, w=None, eps=1e-5, groups=1, gate_first=True):
    """out for [..., dim] inputs."""
    x, z = _split(_f64(x), groups), _split(_f64(z), groups)
    gate = z * _sigmoid(z)
    ww = np.ones(1) if w is None else _f64(w).reshape(groups, -1)
    if gate_first:
        v = x * gate
        out = v * _rstd(v, eps) * ww
    else:
        out = x * _rstd(x, eps) * ww * gate
    return out.reshape(*out.shape[:-2], -1)


def gated_bwd(x, z, w, dout, eps=1e-5, groups=1, gate_first=True):
    """dict of dx, dz, dweight and their terms for [rows, dim] inputs."""
    x, z, dout = (_split(_f64(a), groups) for a in (x, z, dout))
    sg = _sigmoid(z)
    gate, slope = z * sg, sg * (1.0 + z * (1.0 - sg))
    slope_terms = sg * (1.0 + np.abs(z) * (1.0 - sg))
    ww = np.ones(1) if w is None else _f64(w).reshape(groups, -1)
    v = x * gate if gate_first else x
    r = _rstd(v, eps)
    dn = dout if gate_first else dout * gate      # gradient of the normed, weighted value
    g = dn * ww
    dv = r * (g - v * r * r * np.mean(g * v, axis=-1, keepdims=True))
    dvt = r * (np.abs(g) + np.abs(v) * r * r * np.mean(np.abs(g * v), axis=-1, keepdims=True))
    if gate_first:
        dx, dz = dv * gate, dv * x * slope
        dxt, dzt = dvt * np.abs(gate), dvt * np.abs(x) * slope_terms
    else:
        dx, dz = dv, dout * ww * v * r * slope
        dxt, dzt = dvt, np.abs(dout * ww * v * r) * slope_terms
    t = dn * v * r
    flat = lambda a: a.reshape(a.shape[0], -1)  # noqa: E731
    return dict(dx=flat(dx), dz=flat(dz), dx_terms=flat(dxt), dz_terms=flat(dzt), dweight=t.sum(0).reshape(-1),
                dweight_terms=np.abs(t).sum(0).reshape(-1))


def embed_fwd(ids, w, scale=1.0):
    ids, w = np.asarray(ids).astype(np.int64), _f64(w)
    ok = (ids >= 0) & (ids < w.shape[0])
    return np.where(ok[..., None], scale * w[np.where(ok, ids, 0)], 0.0)


def embed_bwd(ids, dout, vocab, scale=1.0, base=None, padding_idx=None):
    """(dweight, terms)."""
    ids = np.asarray(ids).astype(np.int64).reshape(-1)
    dout = _f64(dout).reshape(ids.size, -1)
    ok = (ids >= 0) & (ids < vocab)
    if padding_idx is not None:
        ok &= ids != padding_idx
    dw = np.zeros((vocab, dout.shape[1]))
    terms = np.zeros_like(dw)
    np.add.at(dw, ids[ok], scale * dout[ok])
    np.add.at(terms, ids[ok], np.abs(scale * dout[ok]))
    if base is not None:
        dw += _f64(base)
        terms += np.abs(_f64(base))
    return dw, terms


def grad_norm(tensors):
    return float(np.sqrt(sum(np.sum(_f64(t) ** 2) for t in tensors)))


def grad_clip(tensors, max_norm, eps=1e-6):
    """(norm, the scaled tensors)."""
    n = grad_norm(tensors)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.float64(max_norm) / (np.float64(n) + eps)
    c = 1.0 if q >= 1.0 else q
    with np.errstate(invalid="ignore"):
        return n, [c * _f64(t) for t in tensors]
