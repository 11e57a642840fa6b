"""The gated feed-forward block on the GPU against its definition in fp64.

Bounds.  A product of k terms in fp32 is off by at most k u of the sum of the terms' magnitudes in
any order; the errors are random, so that 8 sqrt(k) u holds with a wide margin, and min(k, ..) for
few terms.  The backward rounds dG and dU to the type of the operands (half a step, relative to each
value) before their products, whose terms they are."""
import numpy as np
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402
from oracle import block  # noqa: E402

from block_helpers import DTYPES, U32, U_OUT, normal, values, within  # noqa: E402

# (tokens, dim, hidden): one of everything, tokens of the skinny kernels and around them, widths
# that no stage, vector or tile divides, several tiles in each direction
SHAPES = [(1, 1, 1), (1, 64, 64), (2, 33, 5), (3, 7, 100), (8, 768, 200), (16, 128, 48),
          (17, 72, 130), (33, 64, 16), (64, 200, 97), (65, 96, 33), (100, 520, 300),
          (129, 64, 257), (300, 128, 128), (257, 1000, 70), (130, 31, 1025), (520, 192, 640)]


def sums(k):
    return min(k, 8.0 * np.sqrt(k)) + 2.0


def _inputs(shape, dtype):
    m, d, f = shape
    return (normal((m, d), dtype, 1), normal((f, d), dtype, 2, d ** -0.5),
            normal((f, d), dtype, 3, d ** -0.5))


def _products(x, wg, wu):
    """G, U and what their errors are at most, in units of the roundoff."""
    g, u = x @ wg.T, x @ wu.T
    k = sums(x.shape[1])
    return g, u, k * (np.abs(x) @ np.abs(wg).T), k * (np.abs(x) @ np.abs(wu).T)


def _slope_max(gelu):
    return 1.2  # |act'| of both stays below


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype, act):
    log(f"mlp forward {shape} {dtype} {act}")
    x, wg, wu = _inputs(shape, dtype)
    out = msel.msel_gated_mlp_fwd(x, wg, wu, act)
    v = [values(t) for t in (x, wg, wu)]
    g, u, eg, eu = _products(*v)
    a = block.act(g, act == "gelu")[0]
    # the activation itself: its exponent is off by a few roundings of its size
    ea = 1.2 * eg + np.abs(a) * (4 * np.abs(g) + 4 * np.abs(g) ** 3 + 16)
    within("out", out, a * u, ea * np.abs(u) + np.abs(a) * eu + 4 * np.abs(a * u))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype, act):
    log(f"mlp backward {shape} {dtype} {act}")
    x, wg, wu = _inputs(shape, dtype)
    dout = normal((shape[0], shape[2]), dtype, 4)
    r = msel.msel_gated_mlp_bwd(x, wg, wu, dout, act)
    vx, vg, vu, vd = (values(t) for t in (x, wg, wu, dout))
    ref = block.mlp_bwd(vx, vg, vu, vd, act == "gelu")
    g, u, eg, eu = _products(vx, vg, vu)
    a, s = block.act(g, act == "gelu")
    near = 4 * np.abs(g) + 4 * np.abs(g) ** 3 + 16
    # errors of dG and dU in units of the roundoff: those of G (|act''| < 1.2), of U, and of their
    # own rounding to the operands' type
    half = U_OUT[DTYPES[dtype]] / U32
    edg = np.abs(vd) * (np.abs(u) * (1.2 * eg + near * (np.abs(s) + 1)) + np.abs(s) * eu) \
        + half * np.abs(ref["dg"])
    edu = np.abs(vd) * (1.2 * eg + np.abs(a) * near) + half * np.abs(ref["du"])
    adg, adu = np.abs(ref["dg"]), np.abs(ref["du"])
    within("dx", r["dx"], ref["dx"], edg @ np.abs(vg) + edu @ np.abs(vu)
           + sums(2 * shape[2]) * (adg @ np.abs(vg) + adu @ np.abs(vu)))
    k = sums(shape[0])
    within("dw_gate", r["dw_gate"], ref["dwg"], (edg + k * adg).T @ np.abs(vx))
    within("dw_up", r["dw_up"], ref["dwu"], (edu + k * adu).T @ np.abs(vx))
    # what is asked for alone is the same
    one = msel.msel_gated_mlp_bwd(x, wg, wu, dout, act, want_dweights=False)
    assert one["dw_gate"] is None and torch.equal(one["dx"], r["dx"])
    other = msel.msel_gated_mlp_bwd(x, wg, wu, dout, act, want_dx=False)
    assert other["dx"] is None and torch.equal(other["dw_up"], r["dw_up"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(5000, 256, 1900), (2100, 520, 3100), (4097, 64, 4100)])
def test_many_tiles(shape, dtype):
    """Enough tiles for the widest ones, with ragged borders; against fp64 on the GPU."""
    log(f"mlp many tiles {shape} {dtype}")
    x, wg, wu = _inputs(shape, dtype)
    out = msel.msel_gated_mlp_fwd(x, wg, wu)
    X, G, U = x.double(), wg.double(), wu.double()
    g, u = X @ G.T, X @ U.T
    s = torch.sigmoid(g)
    k = sums(shape[1])
    eg, eu = k * (X.abs() @ G.abs().T), k * (X.abs() @ U.abs().T)
    ref = g * s * u

    def check(name, got, want, err):
        room = U_OUT[got.dtype] * 1.001 * want.abs() + U32 * err
        worst = float(((got.double() - want).abs() / room).max())
        assert worst <= 1.0, (name, worst)
    near = 4 * g.abs() + 16
    check("out", out, ref, (1.2 * eg + (g * s).abs() * near) * u.abs() + (g * s).abs() * eu
          + 4 * ref.abs())
    dout = normal((shape[0], shape[2]), dtype, 4)
    r = msel.msel_gated_mlp_bwd(x, wg, wu, dout)
    D = dout.double()
    slope = s * (1 + g * (1 - s))
    dg, du = D * u * slope, D * g * s
    half = U_OUT[DTYPES[dtype]] / U32
    edg = D.abs() * (u.abs() * (1.2 * eg + near * (slope.abs() + 1)) + slope.abs() * eu) \
        + half * dg.abs()
    edu = D.abs() * (1.2 * eg + (g * s).abs() * near) + half * du.abs()
    check("dx", r["dx"], dg @ G + du @ U, edg @ G.abs() + edu @ U.abs()
          + sums(2 * shape[2]) * (dg.abs() @ G.abs() + du.abs() @ U.abs()))
    k = sums(shape[0])
    check("dw_gate", r["dw_gate"], dg.T @ X, (edg + k * dg.abs()).T.contiguous() @ X.abs())
    check("dw_up", r["dw_up"], du.T @ X, (edu + k * du.abs()).T.contiguous() @ X.abs())


@pytest.mark.parametrize("tokens", [1, 5, 20, 70, 300])
def test_a_token_is_its_own(tokens):
    """A NaN in one token reaches that token's row alone; leading axes are tokens."""
    log(f"mlp rows {tokens}")
    x, wg, wu = _inputs((tokens, 72, 90), "bf16")
    clean = msel.msel_gated_mlp_fwd(x, wg, wu)
    assert torch.equal(msel.msel_gated_mlp_fwd(x.view(1, tokens, 72), wg, wu)[0], clean)
    x[tokens // 2, 5] = float("nan")
    out = msel.msel_gated_mlp_fwd(x, wg, wu)
    assert torch.isnan(out[tokens // 2]).all()
    keep = torch.arange(tokens, device="cuda") != tokens // 2
    assert torch.equal(out[keep], clean[keep])


def test_refusals():
    x, wg, wu = _inputs((4, 16, 8), "f32")
    dout = torch.zeros(4, 8, device="cuda")
    bad = [lambda: msel.msel_gated_mlp_fwd(x.cpu(), wg, wu),
           lambda: msel.msel_gated_mlp_fwd(x, wg, wu[:4]),
           lambda: msel.msel_gated_mlp_fwd(x, wg.T, wu.T),
           lambda: msel.msel_gated_mlp_fwd(x.bfloat16(), wg, wu),
           lambda: msel.msel_gated_mlp_fwd(x.half(), wg.half(), wu.half()),
           lambda: msel.msel_gated_mlp_fwd(x, wg, None),
           lambda: msel.msel_gated_mlp_fwd(x, wg, wu, "relu"),
           lambda: msel.msel_gated_mlp_fwd(x[:0], wg, wu),
           lambda: msel.msel_gated_mlp_fwd(x[:, ::2], wg[:, :8].contiguous(), wu[:, :8].contiguous()),
           lambda: msel.msel_gated_mlp_fwd(x, wg, wu, out=dout[:3]),
           lambda: msel.msel_gated_mlp_bwd(x, wg, wu, None),
           lambda: msel.msel_gated_mlp_bwd(x, wg, wu, dout[:, :4]),
           lambda: msel.msel_gated_mlp_bwd(x, wg, wu, dout, want_dx=False, want_dweights=False)]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            f()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("size", [30.0, 1e15, 1e21])
def test_gates_far_out(act, size):
    """Where the gate is saturated its slope is 1 or 0, however large its argument: one input, a
    hidden unit for each sign, and nothing added or lost."""
    x = torch.tensor([[size]], device="cuda")
    wg = torch.tensor([[1.0], [-1.0]], device="cuda")
    wu = torch.full((2, 1), 2.0 ** -40, device="cuda")
    dout = torch.ones((1, 2), device="cuda")
    u = size * 2.0 ** -40
    out = msel.msel_gated_mlp_fwd(x, wg, wu, act)
    assert out[0, 0].item() == pytest.approx(size * u, rel=1e-6) and abs(out[0, 1].item()) < 1e-8
    g = msel.msel_gated_mlp_bwd(x, wg, wu, dout, act)
    # dx = dG wg + dU wu = u + size 2^-40, dw_gate = u x for the open unit and 0 for the closed one
    assert g["dx"].item() == pytest.approx(2 * u, rel=1e-6)
    for k, v in (("dw_gate", u * size), ("dw_up", size * size)):
        if v < 3e38:
            assert g[k][0].item() == pytest.approx(v, rel=1e-6)
        assert abs(g[k][1].item()) < 1e-7 * max(1.0, size)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("shape", [(1, 160, 4792), (4, 2088, 40), (7, 128, 40), (31, 129, 130),
                                   (70, 58, 300), (130, 1, 700), (4000, 300, 1)])
def test_gradients_of_few_elements_are_as_good_as_unrounded(shape, act):
    """dG and dU as two bf16 numbers each: the first is off by 2^-8 of the value at most, the second
    is what the first left, off by 2^-8 of that, so that 2^-16 is left of the value (256 roundoffs
    of fp32)."""
    log(f"mlp few elements {shape} {act}")
    x, wg, wu = _inputs(shape, "bf16")
    dout = normal((shape[0], shape[2]), "bf16", 4)
    r = msel.msel_gated_mlp_bwd(x, wg, wu, dout, act)
    vx, vg, vu, vd = (values(t) for t in (x, wg, wu, dout))
    ref = block.mlp_bwd(vx, vg, vu, vd, act == "gelu")
    g, u, eg, eu = _products(vx, vg, vu)
    a, s = block.act(g, act == "gelu")
    near = 4 * np.abs(g) + 4 * np.abs(g) ** 3 + 16
    adg, adu = np.abs(ref["dg"]), np.abs(ref["du"])
    edg = np.abs(vd) * (np.abs(u) * (1.2 * eg + near * (np.abs(s) + 1)) + np.abs(s) * eu) + 256 * adg
    edu = np.abs(vd) * (1.2 * eg + np.abs(a) * near) + 256 * adu
    # the sums have twice the terms; the second ones are 2^-8 of the first
    within("dx", r["dx"], ref["dx"], edg @ np.abs(vg) + edu @ np.abs(vu)
           + sums(4 * shape[2]) * (adg @ np.abs(vg) + adu @ np.abs(vu)))
    k = sums(2 * shape[0])
    within("dw_gate", r["dw_gate"], ref["dwg"], (edg + k * adg).T @ np.abs(vx))
    within("dw_up", r["dw_up"], ref["dwu"], (edu + k * adu).T @ np.abs(vx))


@pytest.mark.parametrize("tokens", [60, 300])
def test_long_sums_in_fp32(tokens):
    """A sum of 4096 products in parts of 512, two products a rounding.  A part's roundings are u / sqrt 3
    of a running sum that grows as a random walk: sqrt(256 / 2) of them, 6.5 u of the part, and so of the
    whole, whose 8 parts' roundings add in squares; 1.2 u for adding them.  Two such factors and
    some roundings of the activation: 10 u of the result's norm.  (In one row it is 27.)"""
    x, wg, wu = _inputs((tokens, 4096, 200), "f32")
    out = msel.msel_gated_mlp_fwd(x, wg, wu)
    X, G, U = x.double(), wg.double(), wu.double()
    g = X @ G.T
    ref = g * torch.sigmoid(g) * (X @ U.T)
    assert float((out.double() - ref).norm() / ref.norm()) <= 14 * U32


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(50, 2048, 130), (200, 1000, 70), (90, 1032, 65), (60, 777, 33),
                                   (130, 4096, 5), (5, 900, 700)])
def test_long_rows_of_few_columns(shape, dtype, act):
    """So few tiles that both projections' sums are split over blocks, with whole and partial last
    stages, and hidden widths that no vector divides."""
    test_forward(shape, dtype, act)
    test_backward(shape, dtype, act)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(200, 1000, 70), (60, 1032, 65), (40, 777, 130), (300, 72, 520),
                                   (700, 200, 1100)])
def test_what_is_not_finite_stays_where_it_belongs(shape, dtype, bad):
    """A token that is not finite changes nothing in the other tokens' rows, and a hidden unit's weights
    nothing in the other units' columns and gradients, at sizes with partial tiles, stages and parts:
    what pads them must not meet it."""
    log(f"mlp not finite {shape} {dtype} {bad}")
    m, d, f = shape
    x, wg, wu = _inputs(shape, dtype)
    dout = normal((m, f), dtype, 4)
    out = msel.msel_gated_mlp_fwd(x, wg, wu)
    clean = msel.msel_gated_mlp_bwd(x, wg, wu, dout)
    for token in (0, m - 1):
        y = x.clone()
        y[token, d - 1] = bad
        others = torch.arange(m, device="cuda") != token
        assert torch.equal(msel.msel_gated_mlp_fwd(y, wg, wu)[others], out[others])
        assert torch.equal(msel.msel_gated_mlp_bwd(y, wg, wu, dout)["dx"][others], clean["dx"][others])
    for unit in (0, f - 1):
        w = wg.clone()
        w[unit, d - 1] = bad
        others = torch.arange(f, device="cuda") != unit
        assert torch.equal(msel.msel_gated_mlp_fwd(x, w, wu)[:, others], out[:, others])
        g = msel.msel_gated_mlp_bwd(x, w, wu, dout, want_dx=False)
        for k in ("dw_gate", "dw_up"):
            assert torch.equal(g[k][others], clean[k][others]), k
