"""The gradient norm over many tensors and clipping on the GPU against the fp64 oracle: mixed
dtypes, odd and empty tensors, element-aligned data, more tensors than one launch takes, lists
whose chunks are cut, in place and into other tensors, values whose squares leave fp32's range,
norms that are zero, infinite and not a number.

Bounds: the sum is fp64, so the norm is off by its rounding to fp32 (u) and a scaled value by
the norm's, the factor's and its own rounding: 4 u, and the rounding of a bf16 output."""
import numpy as np
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402
from selective_state_space_26_amd import _lib  # noqa: E402

from lm_helpers import U32, U_OUT, host, normal  # noqa: E402
from oracle import lm  # noqa: E402


def _check(tensors, max_norm, eps=1e-6):
    n, want = lm.grad_clip([host(t) for t in tensors], max_norm, eps)
    assert abs(float(msel.msel_grad_norm(tensors)) - n) <= 2 * U32 * n
    out = [torch.full_like(t, 7.0) for t in tensors]
    keep = [t.clone() for t in tensors]
    got = msel.msel_grad_clip(msel.GradList(tensors), max_norm, eps, out=out)
    assert abs(float(got) - n) <= 2 * U32 * n
    for t, k, o, w in zip(tensors, keep, out, want):
        assert torch.equal(t, k)
        bound = (U_OUT[t.dtype] * 1.001 + 4 * U32) * np.abs(w) + 1e-44
        assert np.all(np.abs(host(o) - w) <= bound)
    msel.msel_grad_clip(tensors, max_norm, eps)
    for t, o in zip(tensors, out):
        assert torch.equal(t, o)


LISTS = {
    "one": [(1,)], "vector": [(3, 1000)], "empty": [(0,), (5,), (0, 3)],
    "odd": [(7,), (63, 63), (1,), (4097,), (16, 1, 3)],
    "chunks": [(8192,), (4096,), (4095,), (4097,), (100000,)],
    "large": [(1 << 24,), (9999, 1000)],
    "many": [(i % 37 + 1, 3) for i in range(300)],
}


@pytest.mark.parametrize("kind", LISTS)
@pytest.mark.parametrize("dtypes", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip(kind, dtypes, max_norm):
    log(f"clip {kind} {dtypes} {max_norm}")
    dt = (lambda i: ("f32", "bf16")[i % 2]) if dtypes == "mixed" else (lambda i: dtypes)
    tensors = [normal(s, dt(i), i) for i, s in enumerate(LISTS[kind])]
    _check(tensors, max_norm)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clip_element_aligned_views(dtype):
    """Views into one buffer at every alignment."""
    log(f"clip views {dtype}")
    flat = normal((70000,), dtype, 1)
    tensors, at = [], 1
    for n in (1, 2, 3, 1000, 5001, 8, 40001):
        tensors.append(flat[at:at + n])
        at += n + 1
    edge = [flat[0].clone(), flat[at:].clone()]
    _check(tensors, 0.5)
    assert torch.equal(flat[0], edge[0]) and torch.equal(flat[at:], edge[1])


@pytest.mark.parametrize("value", [1e25, 1e-30])
def test_norm_outside_fp32_squares(value):
    """Values whose squares overflow or vanish in fp32."""
    log(f"grad norm of {value}")
    t = [torch.full((5000,), value, device="cuda"), torch.full((3,), value, device="cuda")]
    n = lm.grad_norm([host(x) for x in t])
    assert abs(float(msel.msel_grad_norm(t)) - n) <= 2 * U32 * n


def test_clip_zero_infinite_and_nan():
    log("clip special norms")
    z = [torch.zeros(100, device="cuda")]
    assert float(msel.msel_grad_clip(z, 1.0)) == 0.0 and not z[0].any()
    t = [normal((300,), "f32", 1), normal((50,), "bf16", 2)]
    t[0][7] = float("inf")
    assert float(msel.msel_grad_clip(t, 1.0)) == float("inf")
    assert torch.isnan(t[0][7]) and int(torch.isnan(t[0]).sum()) == 1 and not t[1].any()
    t = [normal((300,), "f32", 1), normal((50,), "bf16", 2)]
    t[1][3] = float("nan")
    assert np.isnan(float(msel.msel_grad_clip(t, 1.0)))
    assert all(torch.isnan(x).all() for x in t)


def test_clip_is_deterministic():
    log("clip determinism")
    t = [normal((100003,), "f32", i) for i in range(5)]
    a, b = msel.msel_grad_norm(t), msel.msel_grad_norm(t)
    assert torch.equal(a, b)


@pytest.mark.parametrize("bad", ["none", "cpu", "dtype", "strided", "count", "sizes", "kinds",
                                 "bound"])
def test_clip_refusals(bad):
    t = [normal((4, 8), "f32", 1), normal((5,), "f32", 2)]
    with pytest.raises((TypeError, ValueError, _lib.MselError)):
        if bad == "none":
            msel.msel_grad_norm([])
        elif bad == "cpu":
            msel.msel_grad_norm([t[0], t[1].cpu()])
        elif bad == "dtype":
            msel.msel_grad_norm([t[0].half()])
        elif bad == "strided":
            msel.msel_grad_norm([t[0].t()])
        elif bad == "count":
            msel.msel_grad_clip(t, 1.0, out=t[:1])
        elif bad == "sizes":
            msel.msel_grad_clip(t, 1.0, out=[t[1], t[0]])
        elif bad == "kinds":
            msel.msel_grad_clip(t, 1.0, out=[x.bfloat16() for x in t])
        else:
            msel.msel_grad_clip(t, -1.0)
