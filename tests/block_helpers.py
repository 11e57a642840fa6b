"""Shared helpers of the tests of the gated recurrence, the log probabilities and the feed-forward
block: a result against the oracle's, within the oracle's bound on the roundings of a computation
in fp32 and half a step of the output's type."""
from __future__ import annotations

import numpy as np
import torch

from lm_helpers import DTYPES, U32, U_OUT, host, normal  # noqa: F401


def within(name, got, ref, err, least=1e-30):
    """|got - ref| <= u_out |ref| + u err (+ least, where results vanish below fp32's range)."""
    g, ref = host(got), np.asarray(ref)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(g[~fine], ref[~fine]), f"{name}: other infinities"
    assert np.all(np.isfinite(g[fine])), f"{name}: non-finite"
    if not fine.any():
        return
    room = (U_OUT[got.dtype] * 1.001 * np.abs(ref) + U32 * np.broadcast_to(err, ref.shape)
            + least)[fine]
    off = np.abs(g[fine] - ref[fine]) / room
    assert off.max() <= 1.0, f"{name}: {off.max():.2f} of the bound"


def values(t):
    """A tensor's values in fp64 on the host, as the oracle takes them."""
    return None if t is None else host(t)
