"""What pins the oracle of the gated recurrence, the log probabilities and the feed-forward block:
closed forms, and the gradients against central differences (CPU)."""
import numpy as np
import pytest

from oracle import block


def _differences(f, v, step=1e-6):
    """df/dv of a scalar function, element by element."""
    g = np.empty_like(v)
    for i in np.ndindex(v.shape):
        keep = v[i]
        v[i] = keep + step
        up = f()
        v[i] = keep - step
        g[i] = (up - f()) / (2 * step)
        v[i] = keep
    return g


def _near(a, b, tol=2e-7):
    # a difference of step 1e-6 is off by step^2 times a third derivative of order one and by
    # eps |f| / step, some 1e-9
    assert np.max(np.abs(a - b)) <= tol * max(1.0, np.max(np.abs(b)))


@pytest.fixture
def rng():
    return np.random.default_rng(5)


def test_lru_closed_forms():
    # an open gate with a constant input: h_t = m sigmoid(gx) x (1 - a^(t+1)) / (1 - a)
    lam = np.array([-0.3])
    ga = np.full((1, 1, 50), 40.0)
    f = block.lru_fwd(np.ones((1, 1, 50)), ga, np.zeros((1, 1, 50)), lam)
    a = np.exp(-0.3)
    t = np.arange(1, 51)
    assert np.allclose(f["out"][0, 0], 0.5 * np.sqrt(1 - a * a) * (1 - a ** t) / (1 - a))
    # a closed one keeps the state and takes nothing in
    f = block.lru_fwd(np.ones((1, 1, 9)), np.full((1, 1, 9), -800.0), np.zeros((1, 1, 9)), lam,
                      np.array([[2.5]]))
    assert np.array_equal(f["out"][0, 0], np.full(9, 2.5))


def test_lru_gradients(rng):
    x, ga, gx, dout = (rng.standard_normal((2, 3, 7)) for _ in range(4))
    lam, h0, df = -np.abs(rng.standard_normal(3)), rng.standard_normal((2, 3)), \
        rng.standard_normal((2, 3))

    def loss():
        f = block.lru_fwd(x, ga, gx, lam, h0)
        return (f["out"] * dout).sum() + (f["final"] * df).sum()
    g = block.lru_bwd(x, ga, gx, lam, dout, h0, df)
    for name, v in (("dx", x), ("dga", ga), ("dgx", gx), ("dlam", lam), ("dh0", h0)):
        _near(_differences(loss, v), g[name])


def test_logprob_closed_forms():
    f = block.logprob_fwd(np.array([[0.0, 0.0, -np.inf, 0.0], [-np.inf] * 4, [3.0] * 4]),
                          np.array([0, 1, 7]), 2.0, 3)
    assert np.allclose(f["logprob"], [-np.log(3), -np.inf, 0.0])
    assert np.allclose(f["lse"], [np.log(3), -np.inf, 6 + np.log(4)])
    assert np.allclose(f["entropy"], [np.log(3), 0.0, np.log(4)])
    assert f["top_ids"].tolist() == [[0, 1, 3], [0, 1, 2], [0, 1, 2]]


def test_logprob_gradients(rng):
    x, ids = rng.standard_normal((4, 6)) * 2, np.array([1, 5, -100, 0])
    dlp, dl, dh = (rng.standard_normal(4) for _ in range(3))

    def loss():
        f = block.logprob_fwd(x, ids, 0.7)
        return (f["logprob"] * dlp + f["lse"] * dl + f["entropy"] * dh).sum()
    _near(_differences(loss, x), block.logprob_bwd(x, ids, 0.7, dlp, dl, dh)[0])


@pytest.mark.parametrize("gelu", [False, True])
def test_mlp_gradients(rng, gelu):
    x, wg, wu = rng.standard_normal((3, 5)), rng.standard_normal((4, 5)), \
        rng.standard_normal((4, 5))
    dout = rng.standard_normal((3, 4))

    def loss():
        return (block.mlp_fwd(x, wg, wu, gelu) * dout).sum()
    g = block.mlp_bwd(x, wg, wu, dout, gelu)
    for name, v in (("dx", x), ("dwg", wg), ("dwu", wu)):
        _near(_differences(loss, v), g[name])
