"""The gated norm over [batch, dim, seqlen] against its definition in fp64, element by element,
computed on the GPU a slice of tokens at a time: for tensors that would take the host too long.
Bounds: lm_helpers."""
from __future__ import annotations

import torch

import selective_state_space_26_amd as msel

from lm_helpers import DTYPES, U32, U_OUT

EPS = 1e-5
SLICE = 512


def uniform(shape, dtype, seed, lo=-1.0, hi=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda", dtype=DTYPES[dtype]).uniform_(lo, hi, generator=g)


def _bound(got, ref, size, what):
    """Element by element, as lm_helpers.assert_elementwise."""
    room = U_OUT[got.dtype] * 1.001 * ref.abs() + 128.0 * U32 * size + 1e-37
    off = (got.double() - ref).abs() / room
    worst = float(off.max())
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound"  # also false for NaN


def _groups(t, groups, bld):
    """A slice of tokens as [batch, groups, n, tokens] in fp64."""
    t = t.transpose(1, 2) if bld else t
    return t.double().reshape(t.shape[0], groups, -1, t.shape[2])


def _cut(t, bld, a, b):
    return t[:, a:b] if bld else t[:, :, a:b]


def inputs(bsz, groups, n, L, dtype):
    shape = (bsz, groups * n, L)
    return (uniform(shape, dtype, 1), uniform(shape, dtype, 2, -4.0, 4.0),
            uniform((groups * n,), "f32", 3, 0.5, 1.5))


def _gate(z):
    s = torch.sigmoid(z)
    return z * s, s * (1.0 + z * (1.0 - s)), s * (1.0 + z.abs() * (1.0 - s))


def check_forward(case, first, out_bld):
    """Returns the bytes of out."""
    bsz, groups, n, L, dtype = case
    x, z, w = inputs(*case)
    out = msel.msel_gated_norm_fwd(x, z, w, EPS, groups, first, "bdl", "bld" if out_bld else "bdl")
    ww = w.double().reshape(1, groups, n, 1)
    for a in range(0, L, SLICE):
        b = min(L, a + SLICE)
        xs, (gate, _, _) = _groups(x[:, :, a:b], groups, False), _gate(z[:, :, a:b].double())
        gate = gate.reshape(xs.shape)
        v = xs * gate if first else xs
        ref = v * (v.square().mean(2, keepdim=True) + EPS) ** -0.5 * ww
        if not first:
            ref = ref * gate
        got = _cut(out, out_bld, a, b)
        _bound((got.transpose(1, 2) if out_bld else got).reshape(ref.shape), ref, ref.abs(),
               f"out {a}")
    return out.numel() * out.element_size()


def check_backward(case, first, bld):
    """Returns the bytes of dx and dz."""
    bsz, groups, n, L, dtype = case
    x, z, w = inputs(*case)
    dout = uniform((bsz, L, groups * n) if bld else (bsz, groups * n, L), dtype, 4)
    g = msel.msel_gated_norm_bwd(x, z, w, dout, EPS, groups, first, "bdl", "bld" if bld else "bdl")
    ww = w.double().reshape(1, groups, n, 1)
    dw, dw_terms = 0.0, 0.0
    for a in range(0, L, SLICE):
        b = min(L, a + SLICE)
        xs = _groups(x[:, :, a:b], groups, False)
        gate, slope, slope_terms = (t.reshape(xs.shape) for t in _gate(z[:, :, a:b].double()))
        dy = _groups(_cut(dout, bld, a, b), groups, bld)
        v = xs * gate if first else xs
        r = (v.square().mean(2, keepdim=True) + EPS) ** -0.5
        p = dy * ww if first else dy * ww * gate
        dv = r * (p - v * r * r * (p * v).mean(2, keepdim=True))
        dvt = r * (p.abs() + v.abs() * r * r * (p * v).abs().mean(2, keepdim=True))
        if first:
            dx, dz, t = dv * gate, dv * xs * slope, dy * v * r
            dxt, dzt = dvt * gate.abs(), dvt * xs.abs() * slope_terms
        else:
            dx, dz, t = dv, dy * ww * v * r * slope, dy * gate * v * r
            dxt, dzt = dvt, (dy * ww * v * r).abs() * slope_terms
        _bound(g["dx"][:, :, a:b].reshape(dx.shape), dx, dxt, f"dx {a}")
        _bound(g["dz"][:, :, a:b].reshape(dz.shape), dz, dzt, f"dz {a}")
        dw = dw + t.sum((0, 3)).reshape(-1)
        dw_terms = dw_terms + t.abs().sum((0, 3)).reshape(-1)
    off = float(((g["dweight"].double() - dw).abs() / (128.0 * U32 * dw_terms)).max())
    assert off <= 1.0, f"dweight: {off:.2f} of the bound"
    return 2 * x.numel() * x.element_size()
