"""What pins the fp64 oracle of the operators around the scan (oracle/lm.py) on the CPU: closed
forms on small inputs, and every gradient against central differences of its forward."""
import numpy as np
import pytest

from oracle import lm


def _r(*shape, seed=0):
    return np.random.default_rng([seed, *shape]).standard_normal(shape)


def _fd(f, x, h=1e-6):
    """Central differences of the scalar f at x, element by element."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[i] = h
        g[i] = (f(x + e) - f(x - e)) / (2 * h)
    return g


def _close(a, b):
    np.testing.assert_allclose(a, b, rtol=2e-6, atol=2e-8)


def test_norm_closed_forms():
    x = np.array([[3.0, 4.0]])
    out, s = lm.norm_fwd(x, eps=0.0)
    _close(out, x / np.sqrt(12.5))
    out, s = lm.norm_fwd(x, np.array([2.0, 1.0]), np.array([[1.0, -4.0]]), 0.5, 0.0)
    np.testing.assert_array_equal(s, [[2.5, -2.0]])
    _close(out, s / np.sqrt((6.25 + 4.0) / 2) * [2.0, 1.0])


@pytest.mark.parametrize("dim", [1, 2, 5])
def test_norm_gradients(dim):
    x, res, w = _r(3, dim, seed=1), _r(3, dim, seed=2), _r(dim, seed=3)
    dout, dres = _r(3, dim, seed=4), _r(3, dim, seed=5)
    a, eps = 0.7, 1e-2

    def loss(x, res, w):
        out, s = lm.norm_fwd(x, w, res, a, eps)
        return np.sum(dout * out) + np.sum(dres * s)
    _, s = lm.norm_fwd(x, w, res, a, eps)
    g = lm.norm_bwd(s, w, dout, dres, a, eps)
    _close(g["dx"], _fd(lambda v: loss(v, res, w), x))
    _close(g["dresidual"], _fd(lambda v: loss(x, v, w), res))
    _close(g["dweight"], _fd(lambda v: loss(x, res, v), w))


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("groups", [1, 2])
def test_gated_gradients(first, groups):
    dim, eps = 6, 1e-2
    x, z, w, dout = _r(3, dim, seed=1), _r(3, dim, seed=2), _r(dim, seed=3), _r(3, dim, seed=4)

    def loss(x, z, w):
        return np.sum(dout * lm.gated_fwd(x, z, w, eps, groups, first))
    g = lm.gated_bwd(x, z, w, dout, eps, groups, first)
    _close(g["dx"], _fd(lambda v: loss(v, z, w), x))
    _close(g["dz"], _fd(lambda v: loss(x, v, w), z))
    _close(g["dweight"], _fd(lambda v: loss(x, z, v), w))


def test_gated_orders_and_groups():
    x, z = _r(2, 4, seed=1), _r(2, 4, seed=2)
    gate = z / (1 + np.exp(-z))
    n = lambda v: v / np.sqrt((v * v).mean(-1, keepdims=True))  # noqa: E731
    _close(lm.gated_fwd(x, z, eps=0.0), n(x * gate))
    _close(lm.gated_fwd(x, z, eps=0.0, gate_first=False), n(x) * gate)
    _close(lm.gated_fwd(x, z, eps=0.0, groups=2)[:, :2], n((x * gate)[:, :2]))


def test_embed():
    w, ids = _r(4, 3), np.array([[1, 3, -1], [4, 1, 0]])
    out = lm.embed_fwd(ids, w, 2.0)
    _close(out[0, 0], 2.0 * w[1])
    assert not out[0, 2].any() and not out[1, 0].any()
    dout, base = _r(2, 3, 3, seed=1), _r(4, 3, seed=2)
    dw, _ = lm.embed_bwd(ids, dout, 4, 2.0, base)
    _close(dw - base, _fd(lambda v: np.sum(dout * lm.embed_fwd(ids, v, 2.0)), w))
    dw, _ = lm.embed_bwd(ids, dout, 4, 2.0, padding_idx=1)
    assert not dw[1].any() and not dw[2].any()


def test_clip():
    t = [np.array([3.0, 0.0]), np.array([[4.0]])]
    n, out = lm.grad_clip(t, 1.0, 0.0)
    assert n == 5.0
    _close(out[1], [[0.8]])
    n, out = lm.grad_clip(t, 6.0)
    np.testing.assert_array_equal(out[0], t[0])
    n, out = lm.grad_clip([np.array([np.inf, 1.0])], 1.0)
    assert n == np.inf and np.isnan(out[0][0]) and out[0][1] == 0.0
