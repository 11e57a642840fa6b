"""The gated feed-forward block at sizes that take each of its product kernels' tiles, the widest among
them, against its definition in fp64 on the GPU."""
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402

from selective_state_space_26_amd import _lib  # noqa: E402

from block_helpers import DTYPES, U32, U_OUT, normal  # noqa: E402
from mlp_shapes import LONG_F32, TILES  # noqa: E402


def _inputs(shape, dtype):
    m, d, f = shape
    return (normal((m, d), dtype, 1), normal((f, d), dtype, 2, d ** -0.5),
            normal((f, d), dtype, 3, d ** -0.5), normal((m, f), dtype, 4))


@pytest.mark.parametrize("shape", LONG_F32)
def test_long_sums_in_fp32_at_every_size(shape):
    """Sums in parts of 512 products whatever the tile.  A part's roundings are 6.5 u of it (256 steps,
    each u / sqrt 3 of a sum that grows as a random walk), and so of the whole; its up to 32 parts add
    sqrt(32 / 2) u / sqrt 3 = 2.3 u.  G and U are each off by 6.9 u, their product by 9.8 u, the
    activation's roundings add 1 or 2; dx and the weights' gradients are sums of such terms (of which the
    errors add in squares, as the terms) with roundings of their own: sqrt(9.8^2 + 6.9^2) = 12 u of the
    result's norm.  (In one running sum of 4096 or 16384 products it is 23 to 29.)"""
    log(f"mlp long fp32 sums {shape}")
    x, wg, wu, dout = _inputs(shape, "f32")
    X, G, W, D = (t.double() for t in (x, wg, wu, dout))
    g, u = X @ G.T, X @ W.T
    s = torch.sigmoid(g)

    def check(name, got, ref):
        off = float((got.double() - ref).norm() / ref.norm()) / U32
        assert off <= 14, (name, off)
    check("out", msel.msel_gated_mlp_fwd(x, wg, wu), g * s * u)
    r = msel.msel_gated_mlp_bwd(x, wg, wu, dout)
    dg, du = D * u * s * (1 + g * (1 - s)), D * g * s
    check("dx", r["dx"], dg @ G + du @ W)
    check("dw_gate", r["dw_gate"], dg.T @ X)
    check("dw_up", r["dw_up"], du.T @ X)


@pytest.mark.parametrize("tokens", [1, 20, 70, 4096, 4097])
@pytest.mark.parametrize("split", [False, True])
def test_gradients_that_round_to_infinity(tokens, split):
    """dU = 181^2 2^113, finite in fp32 and above bf16's largest value by more than half a step: it
    rounds to infinity, whether dG and dU are held in one bf16 number or in two, and so do the sums
    that it is a term of.  dG = dout U act'(G) is 2^-12 of that: finite.  split: rows so long that both
    projections' sums are split over blocks."""
    log(f"mlp gradients beyond bf16 {tokens} {split}")
    dim = 1032 if split else 1
    x = torch.zeros((tokens, dim), device="cuda", dtype=torch.bfloat16)
    wg, wu = (torch.zeros((1, dim), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    dout = torch.zeros((tokens, 1), device="cuda", dtype=torch.bfloat16)
    x[-1, 0], wg[0, 0], wu[0, 0] = 0.5, 181.0, 2.0 ** -11
    dout[-1, 0] = 181.0 * 2.0 ** 114
    r = msel.msel_gated_mlp_bwd(x, wg, wu, dout)
    # G = 90.5, so that act(G) = G and act'(G) = 1 in fp32; U = 2^-12, dG = 181 2^102
    assert torch.equal(r["dw_gate"][0, :1], torch.tensor([181.0 * 2.0 ** 101], device="cuda").bfloat16())
    assert r["dw_up"][0, 0].item() == float("inf")
    assert r["dx"][-1, 0].item() == float("inf")
    assert bool((r["dx"][:-1] == 0).all())


def _act(g, gelu):
    """The activation and its slope in fp64."""
    if not gelu:
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = (2.0 / torch.pi) ** 0.5
    s = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * 2 * c * (1 + 0.134145 * g * g)


def _sums(k):
    return min(k, 8.0 * k ** 0.5) + 2.0


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", TILES)
def test_every_tile_of_every_product(shape, dtype, act):
    """Element by element.  A sum of k products in fp32 is off by at most k u of the sum of their
    magnitudes, 8 sqrt(k) u with a wide margin where the errors are random; |act''| < 1.2; the
    activation's exponent is off by a few roundings of its size, up to 4 (|g| + |g|^3); dG and dU are
    rounded to the type of the operands.  Gradients of few elements have a second number each, so twice
    the terms."""
    log(f"mlp tiles {shape} {dtype} {act}")
    x, wg, wu, dout = _inputs(shape, dtype)
    X, G, W, D = (t.double() for t in (x, wg, wu, dout))
    g, u = X @ G.T, X @ W.T
    a, slope = _act(g, act == "gelu")
    k = _sums(shape[1])
    eg, eu = k * (X.abs() @ G.abs().T), k * (X.abs() @ W.abs().T)
    near = 4 * g.abs() + 4 * g.abs() ** 3 + 16

    def check(name, got, want, err):
        room = U_OUT[got.dtype] * 1.001 * want.abs() + U32 * err
        worst = float(((got.double() - want).abs() / room).max())
        assert worst <= 1.0, (name, worst)
    ea = 1.2 * eg + a.abs() * near
    check("out", msel.msel_gated_mlp_fwd(x, wg, wu, act), a * u,
          ea * u.abs() + a.abs() * eu + 4 * (a * u).abs())
    r = msel.msel_gated_mlp_bwd(x, wg, wu, dout, act)
    dg, du = D * u * slope, D * a
    half = U_OUT[DTYPES[dtype]] / U32
    edg = D.abs() * (u.abs() * (1.2 * eg + near * (slope.abs() + 1)) + slope.abs() * eu) \
        + half * dg.abs()
    edu = D.abs() * ea + half * du.abs()
    k = _sums(4 * shape[2])
    check("dx", r["dx"], dg @ G + du @ W, edg @ G.abs() + edu @ W.abs()
          + k * (dg.abs() @ G.abs() + du.abs() @ W.abs()))
    k = _sums(2 * shape[0])
    check("dw_gate", r["dw_gate"], dg.T @ X, (edg + k * dg.abs()).T @ X.abs())
    check("dw_up", r["dw_up"], du.T @ X, (edu + k * du.abs()).T @ X.abs())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", TILES)
def test_in_range_and_twice_alike(shape, dtype):
    """The checked build counts no index out of its buffer, and it and a second run give the same
    bits."""
    log(f"mlp tiles, checked build {shape} {dtype}")
    x, wg, wu, dout = _inputs(shape, dtype)

    def run():
        return dict(out=msel.msel_gated_mlp_fwd(x, wg, wu, "gelu"),
                    **msel.msel_gated_mlp_bwd(x, wg, wu, dout, "gelu"))
    with _lib.using(_lib.LIB_CHECKED_PATH):
        msel.bound_violations()
        got = run()
        count, f, line = msel.bound_violations()
        assert count == 0, f"{count} out-of-range indexes, the first at {f}:{line}"
    for _ in range(2):
        for k, v in run().items():
            assert torch.equal(v, got[k]), k
