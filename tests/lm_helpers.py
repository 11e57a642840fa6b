"""Shared helpers of the tests of the operators around the scan: seeded tensors on the GPU and
bounds derived from the arithmetic.

Unit roundoffs: u = 2^-24 for fp32 arithmetic, 2^-8 for the rounding of an output to bf16 (24 and
8 bits of significand, round to nearest).

* Elementwise outputs (norms): a value is a product of a few factors, each computed with a few
  roundings, and of rstd, whose sum of squares takes at most 16 + 6 + 16 additions one after
  another in the row kernels (a lane's values, the lanes, the wavefronts) and 16384 / 32 + 6 + 16
  in the strided ones, where the running sum grows evenly, so that its errors add up to less
  than half of their worst case.  128 u of the value's terms (their magnitudes, where they may
  cancel) covers these with the exp and the reciprocal of the gate: the relative error of a sum
  of squares is halved by the root.
* Sums over many rows (dweight, the embedding's gradient): at most about 1100 terms are added one
  after another, but each addition's error is u of the partial sum, which stays far below the sum
  of magnitudes except in its last part: 128 u times the sum of the terms' magnitudes.
"""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
U_OUT = {torch.float32: U32, torch.bfloat16: 2.0 ** -8}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def normal(shape, dtype="f32", seed=0, std=1.0, mean=0.0):
    """A seeded tensor on the GPU, drawn on the host."""
    r = np.random.default_rng([seed, *[int(s) for s in shape]])
    x = torch.from_numpy(r.standard_normal(shape, dtype=np.float32) * np.float32(std)
                         + np.float32(mean))
    return x.to(DTYPES[dtype]).cuda()


def host(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def assert_elementwise(name, got, ref, terms=None, k=128.0):
    """|got - ref| <= u_out |ref| + k u terms (|ref| itself unless given), element by element."""
    u = U_OUT[got.dtype]
    g = host(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{name}: non-finite"
    size = np.abs(ref) if terms is None else terms
    bad = np.abs(g - ref) / (u * 1.001 * np.abs(ref) + k * U32 * size + 1e-37)
    at = np.unravel_index(bad.argmax(), bad.shape)
    assert bad.max() <= 1.0, f"{name}: {bad.max():.2f} of the bound at {at}"


def assert_sum(name, got, ref, terms, k=128.0):
    """|got - ref| <= k u (sum of the magnitudes of the terms)."""
    g = host(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{name}: non-finite"
    bad = np.abs(g - ref) / (k * U32 * terms + 1e-37)
    assert bad.max() <= 1.0, f"{name}: {bad.max():.2f} of the bound"
