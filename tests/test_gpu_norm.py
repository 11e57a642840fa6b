"""The norms before and after a block on the GPU against the fp64 oracle: forward and backward,
every dtype pair, layout and gate order, widths around the limits of one, four and sixteen
wavefronts a row and of the tiles, odd widths and lengths, one row, absent optional tensors,
in-place residuals, streams, non-finite rows.  The bounds are derived in lm_helpers."""
import numpy as np
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402
from selective_state_space_26_amd import _lib  # noqa: E402

from lm_helpers import DTYPES, assert_elementwise, assert_sum, host, normal  # noqa: E402
from oracle import lm  # noqa: E402

PAIRS = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]
# widths: one element, less than a vector, a vector and its neighbours, the last width of 16 lanes
# a row (64 and 128) and the next, of one vector per lane of a wavefront (256 and 512), of four
# (1024 and 2048), of four wavefronts (4096, 8192), the largest
DIMS = [1, 3, 7, 8, 63, 64, 65, 128, 131, 255, 257, 512, 513, 768, 1023, 1024,
        1025, 2048, 2049, 4097, 8192, 8195, 16384]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,rdtype", PAIRS)
def test_norm(dim, dtype, rdtype):
    rows = 9 if dim < 5000 else 3
    log(f"norm {rows}x{dim} {dtype} {rdtype}")
    x, r = normal((rows, dim), dtype, 1), normal((rows, dim), rdtype, 2, 2.0)
    w = normal((dim,), "f32", 3, 0.1, 1.0)
    out, s = msel.msel_norm_fwd(x, w, r, 0.5, 1e-5)
    ro, rs = lm.norm_fwd(host(x), host(w), host(r), 0.5, 1e-5)
    assert s.dtype == DTYPES[rdtype] and out.dtype == DTYPES[dtype]
    assert_elementwise("s", s, rs, k=1.0)
    assert_elementwise("out", out, ro)
    dout, dr = normal((rows, dim), dtype, 4), normal((rows, dim), rdtype, 5)
    g = msel.msel_norm_bwd(s, w, dout, dr, 0.5, 1e-5)
    ref = lm.norm_bwd(host(s), host(w), host(dout), host(dr), 0.5, 1e-5)
    assert_elementwise("dx", g["dx"], ref["dx"], ref["dx_terms"])
    assert_elementwise("dresidual", g["dresidual"], ref["dresidual"], ref["dresidual_terms"])
    assert_sum("dweight", g["dweight"], ref["dweight"], ref["dweight_terms"])


@pytest.mark.parametrize("rows", [1, 2, 5, 2049, 20000])
def test_norm_row_counts(rows):
    """One row, fewer rows than a block has teams, more rows than the grid has teams."""
    dim = 48
    log(f"norm rows {rows}")
    x, w = normal((rows, dim), "bf16", 1), normal((dim,), "f32", 3, 0.1, 1.0)
    r = normal((rows, dim), "f32", 2)
    out, s = msel.msel_norm_fwd(x, w, r)
    ro, rs = lm.norm_fwd(host(x), host(w), host(r))
    assert_elementwise("out", out, ro)
    dout = normal((rows, dim), "bf16", 4)
    g = msel.msel_norm_bwd(s, w, dout)
    ref = lm.norm_bwd(host(s), host(w), host(dout))
    assert_elementwise("dx", g["dx"], ref["dx"], ref["dx_terms"])
    assert_sum("dweight", g["dweight"], ref["dweight"], ref["dweight_terms"])


def test_norm_optional_tensors():
    log("norm optional tensors")
    rows, dim = 6, 100
    x = normal((2, 3, dim), "bf16", 1)
    out, s = msel.msel_norm_fwd(x)
    assert s is None and out.shape == x.shape
    ro, rs = lm.norm_fwd(host(x))
    assert_elementwise("out", out, ro)
    out2, s2 = msel.msel_norm_fwd(x, residual_dtype=torch.float32)
    assert torch.equal(out, out2) and torch.equal(s2, x.float())
    dout = normal((2, 3, dim), "bf16", 4)
    g = msel.msel_norm_bwd(s2, None, dout, want_dresidual=False, want_dweight=False)
    assert g["dresidual"] is None and g["dweight"] is None
    ref = lm.norm_bwd(host(s2).reshape(rows, dim), None, host(dout).reshape(rows, dim))
    assert_elementwise("dx", g["dx"].reshape(rows, dim), ref["dx"], ref["dx_terms"])
    g = msel.msel_norm_bwd(s2, None, dout, want_dx=False)
    assert g["dx"] is None
    assert_elementwise("dresidual", g["dresidual"].reshape(rows, dim), ref["dresidual"],
                       ref["dresidual_terms"])
    assert_sum("dweight", g["dweight"], ref["dweight"], ref["dweight_terms"])


def test_norm_in_place():
    log("norm in place")
    x, r = normal((33, 500), "bf16", 1), normal((33, 500), "f32", 2)
    w = normal((500,), "f32", 3)
    out, s = msel.msel_norm_fwd(x, w, r, 0.25)
    keep = r.clone()
    out2, s2 = msel.msel_norm_fwd(x, w, keep, 0.25, residual_out=keep)
    assert s2 is keep and torch.equal(s2, s) and torch.equal(out, out2)
    dout, dr = normal((33, 500), "bf16", 4), normal((33, 500), "f32", 5)
    g = msel.msel_norm_bwd(s, w, dout, dr, 0.25)
    g2 = msel.msel_norm_bwd(s, w, dout, dr, 0.25, dresidual=dr)
    assert g2["dresidual"] is dr
    for k in g:
        assert torch.equal(g[k], g2[k]), k


LAYOUTS = [("bdl", "bdl"), ("bdl", "bld"), ("bld", "bld")]
# batch, dim, seqlen, groups: one step; less than a vector of tokens; a tile and its neighbours;
# channels around a pass of the tile; odd everything; groups of a few channels; more tiles than
# one batch row; wide
SHAPES = [(3, 24, 1, 1), (2, 5, 3, 1), (1, 1, 40, 1), (50, 70, 8, 1),
          (40, 300, 19, 1), (9, 40, 31, 8), (40, 33, 4, 1), (300, 7, 5, 1), (2, 64, 31, 2),
          (40, 600, 40, 1), (3, 1030, 700, 1), (17, 1040, 70, 2), (37, 5121, 9, 1), (1, 129, 32, 1),
          (2, 130, 33, 1), (1, 1000, 77, 4), (3, 96, 250, 8), (1, 1536, 64, 1), (2, 1537, 70, 1),
          (1, 2050, 65, 2), (1, 5120, 48, 1), (1, 5121, 40, 1), (1, 16384, 36, 1)]


def _to_rows(t, layout):
    a = host(t)
    if layout == "bdl":
        a = a.transpose(0, 2, 1)
    return a.reshape(-1, a.shape[-1])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("layout,out_layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("first", [True, False], ids=["gate_first", "gate_last"])
def test_gated_norm(shape, layout, out_layout, dtype, first):
    bsz, dim, L, groups = shape
    log(f"gated norm {shape} {layout}->{out_layout} {dtype} {'first' if first else 'last'}")
    at = (bsz, dim, L) if layout == "bdl" else (bsz, L, dim)
    to = (bsz, dim, L) if out_layout == "bdl" else (bsz, L, dim)
    x, z = normal(at, dtype, 1), normal(at, dtype, 2)
    w, dout = normal((dim,), "f32", 3, 0.1, 1.0), normal(to, dtype, 4)
    args = (1e-5, groups, first, layout, out_layout)
    out = msel.msel_gated_norm_fwd(x, z, w, *args)
    assert tuple(out.shape) == to
    rx, rz, rd = _to_rows(x, layout), _to_rows(z, layout), _to_rows(dout, out_layout)
    opt = dict(eps=1e-5, groups=groups, gate_first=first)

    def rows(t, lay):
        if lay == "bdl":
            t = t.transpose(1, 2)
        return t.reshape(-1, dim)
    assert_elementwise("out", rows(out, out_layout), lm.gated_fwd(rx, rz, host(w), **opt))
    g = msel.msel_gated_norm_bwd(x, z, w, dout, *args)
    ref = lm.gated_bwd(rx, rz, host(w), rd, **opt)
    assert_elementwise("dx", rows(g["dx"], layout), ref["dx"], ref["dx_terms"])
    assert_elementwise("dz", rows(g["dz"], layout), ref["dz"], ref["dz_terms"])
    assert_sum("dweight", g["dweight"], ref["dweight"], ref["dweight_terms"])


# channels of a group (8 groups, 240 or more wide tiles): every block size, groups held on the CU
# whole and in part
@pytest.mark.parametrize("n", [40, 203, 300, 700, 1001, 1601])
@pytest.mark.parametrize("dtype,first,out_layout", [("bf16", True, "bld"), ("f32", False, "bdl")])
def test_gated_norm_wide_tiles(n, dtype, first, out_layout):
    bsz, groups, L = 1, 8, 1873 if dtype == "bf16" else 937
    dim = groups * n
    log(f"gated norm wide tiles {n} {dtype}")
    x, z = normal((bsz, dim, L), dtype, 1), normal((bsz, dim, L), dtype, 2)
    w = normal((dim,), "f32", 3, 0.1, 1.0)
    dout = normal((bsz, dim, L) if out_layout == "bdl" else (bsz, L, dim), dtype, 4)
    args = (1e-5, groups, first, "bdl", out_layout)
    out = msel.msel_gated_norm_fwd(x, z, w, *args)
    g = msel.msel_gated_norm_bwd(x, z, w, dout, *args)
    opt = dict(eps=1e-5, groups=groups, gate_first=first)
    rx, rz, rd = _to_rows(x, "bdl"), _to_rows(z, "bdl"), _to_rows(dout, out_layout)

    def rows(t, lay):
        return (t.transpose(1, 2) if lay == "bdl" else t).reshape(-1, dim)
    assert_elementwise("out", rows(out, out_layout), lm.gated_fwd(rx, rz, host(w), **opt))
    ref = lm.gated_bwd(rx, rz, host(w), rd, **opt)
    assert_elementwise("dx", rows(g["dx"], "bdl"), ref["dx"], ref["dx_terms"])
    assert_elementwise("dz", rows(g["dz"], "bdl"), ref["dz"], ref["dz_terms"])
    assert_sum("dweight", g["dweight"], ref["dweight"], ref["dweight_terms"])


@pytest.mark.parametrize("layout,out_layout", LAYOUTS)
def test_gated_norm_many_tiles_without_weight(layout, out_layout):
    """More tiles and rows than the backward's grid has blocks; no weight, no dweight."""
    bsz, dim, L = 5, 20, 6007
    log(f"gated norm many tiles {layout} {out_layout}")
    at = (bsz, dim, L) if layout == "bdl" else (bsz, L, dim)
    to = (bsz, dim, L) if out_layout == "bdl" else (bsz, L, dim)
    x, z, dout = normal(at, "bf16", 1), normal(at, "bf16", 2), normal(to, "bf16", 3)
    kw = dict(layout=layout, out_layout=out_layout)
    g = msel.msel_gated_norm_bwd(x, z, None, dout, **kw)
    ref = lm.gated_bwd(_to_rows(x, layout), _to_rows(z, layout), None, _to_rows(dout, out_layout))
    assert_sum("dweight", g["dweight"], ref["dweight"], ref["dweight_terms"])
    dx = g["dx"].transpose(1, 2) if layout == "bdl" else g["dx"]
    assert_elementwise("dx", dx.reshape(-1, dim), ref["dx"], ref["dx_terms"])
    g2 = msel.msel_gated_norm_bwd(x, z, None, dout, want_dweight=False, **kw)
    assert g2["dweight"] is None and torch.equal(g["dx"], g2["dx"]) and torch.equal(g["dz"], g2["dz"])


def test_norms_are_deterministic_and_keep_their_stream():
    log("norm determinism, side stream")
    x, z = normal((2, 300, 1000), "bf16", 1), normal((2, 300, 1000), "bf16", 2)
    dout, w = normal((2, 1000, 300), "bf16", 3), normal((300,), "f32", 4)
    ref = msel.msel_gated_norm_bwd(x, z, w, dout, out_layout="bld")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = msel.msel_gated_norm_bwd(x, z, w, dout, out_layout="bld")
    side.synchronize()
    for k in ref:
        assert torch.equal(ref[k], got[k]), k


def test_norm_nonfinite_rows_stay_in_their_row():
    """A row of NaN or infinity spoils itself alone, and a zero row is all zeros."""
    log("norm non-finite rows")
    x = normal((8, 300), "f32", 1)
    x[2, 17] = float("nan")
    x[4, 299] = float("inf")
    x[6] = 0.0
    out, _ = msel.msel_norm_fwd(x)
    ok = [0, 1, 3, 5, 7]
    ro, _ = lm.norm_fwd(host(x[ok]))
    assert_elementwise("out", out[ok], ro)
    assert torch.isnan(out[2]).all() and torch.isnan(out[4, 299]) and not out[4, :299].any()
    assert not out[6].any()


def test_gated_norm_saturated_gates():
    """Gates far into both tails: silu(-200) is -0 and silu(200) is 200."""
    log("gated norm saturated")
    z = torch.tensor([-200.0, -100.0, -50.0, 0.0, 50.0, 100.0, 200.0, 1.0], device="cuda")
    z = z.repeat(4, 5).reshape(4, 40, 1).repeat(1, 1, 9).contiguous()
    x = normal((4, 40, 9), "f32", 1)
    out = msel.msel_gated_norm_fwd(x, z)
    assert_elementwise("out", out.transpose(1, 2).reshape(-1, 40),
                       lm.gated_fwd(_to_rows(x, "bdl"), _to_rows(z, "bdl")))


@pytest.mark.parametrize("bad", ["cpu", "dtype", "shape", "strided", "weight", "pair", "wide"])
def test_norm_refusals(bad):
    x, r = normal((4, 8), "f32", 1), normal((4, 8), "f32", 2)
    w = normal((8,), "f32", 3)
    err = (TypeError, ValueError, _lib.MselError)
    with pytest.raises(err):
        if bad == "cpu":
            msel.msel_norm_fwd(x.cpu(), w, r)
        elif bad == "dtype":
            msel.msel_norm_fwd(x.half(), w, r)
        elif bad == "shape":
            msel.msel_norm_fwd(x, w, r[:2])
        elif bad == "strided":
            msel.msel_norm_fwd(x.t(), w, r)
        elif bad == "weight":
            msel.msel_norm_fwd(x, w.bfloat16(), r)
        elif bad == "pair":
            msel.msel_norm_fwd(x, w, r.bfloat16())
        else:
            msel.msel_norm_fwd(normal((1, 16385), "f32", 1))


@pytest.mark.parametrize("bad", ["layouts", "turn", "groups", "z", "dout"])
def test_gated_norm_refusals(bad):
    x, z = normal((2, 6, 8), "f32", 1), normal((2, 6, 8), "f32", 2)
    with pytest.raises((TypeError, ValueError, _lib.MselError)):
        if bad == "layouts":
            msel.msel_gated_norm_fwd(x, z, layout="ldb")
        elif bad == "turn":
            msel.msel_gated_norm_fwd(x, z, layout="bld", out_layout="bdl")
        elif bad == "groups":
            msel.msel_gated_norm_fwd(x, z, groups=4)
        elif bad == "z":
            msel.msel_gated_norm_fwd(x, z[:, :, :4])
        else:
            msel.msel_gated_norm_bwd(x, z, None, x, out_layout="bld")
