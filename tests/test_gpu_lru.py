"""The gated linear recurrence on the GPU against its definition in fp64, over every way a row is
worked on: a step, a lane, 16 lanes, a wavefront, four wavefronts, segments."""
import numpy as np
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402
from oracle import block  # noqa: E402

from block_helpers import normal, values, within  # noqa: E402

SHAPES = [(1, 1, 1), (3, 70, 1), (2, 3, 2), (1, 5, 7), (3, 90, 8), (2, 3, 9), (1, 2, 100),
          (3, 37, 128), (1, 3, 129), (2, 2, 511), (2, 2, 512), (1, 3, 513), (1, 1, 2049),
          (5, 130, 600), (1, 515, 4100), (8, 513, 700), (1, 4, 5000), (2, 3, 30011)]


def _inputs(shape, dtype, carried, std=1.5):
    t = dict(x=normal(shape, dtype, 1), gate_a=normal(shape, dtype, 2, std),
             gate_x=normal(shape, dtype, 3, std), lam=-normal(shape[1:2], "f32", 4).abs() * 0.7)
    t["h0"] = normal(shape[:2], "f32", 5) if carried else None
    return t


def _oracle_args(t):
    return [values(t[k]) for k in ("x", "gate_a", "gate_x", "lam")]


@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype, carried):
    log(f"lru forward {shape} {dtype} {carried}")
    t = _inputs(shape, dtype, carried)
    out, final, chunks = msel.msel_lru_fwd(**t, return_chunk_states=True)
    ref = block.lru_fwd(*_oracle_args(t), values(t["h0"]))
    within("out", out, ref["out"], ref["out_err"])
    within("final", final, ref["final"], ref["final_err"])
    T = msel.chunk_len()
    first = values(t["h0"]) if carried else np.zeros(shape[:2])
    states = np.concatenate([first[..., None], ref["out"]], -1)[..., 0:shape[2]:T]
    errs = np.concatenate([0 * first[..., None], ref["out_err"]], -1)[..., 0:shape[2]:T]
    within("chunk_states", chunks, states, errs)


@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype, carried):
    log(f"lru backward {shape} {dtype} {carried}")
    t = _inputs(shape, dtype, carried)
    dout = normal(shape, dtype, 6)
    dfinal = normal(shape[:2], "f32", 7) if carried else None
    ref = block.lru_bwd(*_oracle_args(t), values(dout), values(t["h0"]), values(dfinal))
    chunks = msel.msel_lru_fwd(**t, return_chunk_states=True)[2]
    given = msel.msel_lru_bwd(**t, dout=dout, dfinal_state=dfinal, chunk_states=chunks,
                              want_dh0=True)
    rebuilt = msel.msel_lru_bwd(**t, dout=dout, dfinal_state=dfinal, want_dh0=True)
    for name, key in (("dx", "dx"), ("dgate_a", "dga"), ("dgate_x", "dgx"), ("dlam", "dlam"),
                      ("dh0", "dh0")):
        within(name, given[name], ref[key], ref[key + "_err"])
        assert torch.equal(given[name], rebuilt[name]), name


@pytest.mark.parametrize("shape", [(2, 3, 40), (1, 3, 700), (600, 1, 700)])
def test_open_and_closed_gates(shape):
    """Gates far from 0: a between 0 and 1 exactly, m from 0 on."""
    log(f"lru gates {shape}")
    t = _inputs(shape, "f32", True, std=40.0)
    t["lam"] = t["lam"] * 30.0
    t["lam"][0] = 0.0
    dout = normal(shape, "f32", 6)
    out, final, _ = msel.msel_lru_fwd(**t)
    f = block.lru_fwd(*_oracle_args(t), values(t["h0"]))
    # what a sigmoid below fp32's range would give
    within("out", out, f["out"], f["out_err"], 1e-17)
    g = msel.msel_lru_bwd(**t, dout=dout, want_dh0=True)
    ref = block.lru_bwd(*_oracle_args(t), values(dout), values(t["h0"]))
    for name, key in (("dx", "dx"), ("dgate_a", "dga"), ("dgate_x", "dgx"), ("dlam", "dlam"),
                      ("dh0", "dh0")):
        within(name, g[name], ref[key], ref[key + "_err"], 1e-17)


@pytest.mark.parametrize("shape", [(3, 5, 6), (2, 3, 100), (1, 700, 1500), (2, 3, 9000)])
def test_carried_state_in_place(shape):
    """A sequence in two calls, the state updated in place, equals the one call closely; the first
    part bit for bit where rows are worked on alike."""
    log(f"lru carried {shape}")
    t = _inputs(shape, "f32", True)
    ref = block.lru_fwd(*_oracle_args(t), values(t["h0"]))
    cut = shape[2] // 2
    state, parts = t["h0"].clone(), []
    for a, b in ((0, cut), (cut, shape[2])):
        part = {k: t[k][..., a:b].contiguous() for k in ("x", "gate_a", "gate_x")}
        out, final, _ = msel.msel_lru_fwd(**part, lam=t["lam"], h0=state, final_state=state)
        assert final is state
        parts.append(out)
    within("out", torch.cat(parts, -1), ref["out"], ref["out_err"])
    within("final", state, ref["final"], ref["final_err"])


def test_decode_steps_give_the_sequence():
    log("lru decode")
    t = _inputs((4, 33, 12), "bf16", False)
    whole = msel.msel_lru_fwd(**t)[0]
    state, steps = torch.zeros(4, 33, device="cuda"), []
    for k in range(12):
        part = {n: t[n][..., k:k + 1].contiguous() for n in ("x", "gate_a", "gate_x")}
        steps.append(msel.msel_lru_fwd(**part, lam=t["lam"], h0=state, final_state=state)[0])
    ref = block.lru_fwd(*_oracle_args(t))
    within("steps", torch.cat(steps, -1), ref["out"], ref["out_err"])
    within("whole", whole, ref["out"], ref["out_err"])


@pytest.mark.parametrize("shape", [(2, 3, 20), (1, 3, 700), (520, 1, 3000), (2, 2, 9000)])
def test_what_is_not_finite_stays_in_its_row(shape):
    """NaN and infinite inputs reach the later steps of their row alone; gradients likewise."""
    log(f"lru non-finite {shape}")
    t = _inputs(shape, "f32", True)
    dout = normal(shape, "f32", 6)
    clean = msel.msel_lru_fwd(**t)[0]
    clean_g = msel.msel_lru_bwd(**t, dout=dout)
    k = shape[2] // 2
    t["x"][0, 0, k] = float("nan")
    out = msel.msel_lru_fwd(**t)[0]
    assert torch.isnan(out[0, 0, k:]).all()
    assert torch.equal(out[0, 0, :k], clean[0, 0, :k])
    others = torch.ones(shape[:2], dtype=torch.bool, device="cuda")
    others[0, 0] = False
    assert torch.equal(out[others], clean[others])
    g = msel.msel_lru_bwd(**t, dout=dout)
    for n in ("dx", "dgate_a", "dgate_x"):
        assert torch.equal(g[n][others], clean_g[n][others]), n
    assert torch.equal(g["dx"][0, 0, :k], clean_g["dx"][0, 0, :k])


def test_a_positive_rate_is_nan():
    t = _inputs((1, 2, 30), "f32", False)
    t["lam"][0] = 0.5
    out = msel.msel_lru_fwd(**t)[0]
    assert torch.isnan(out[0, 0]).all() and torch.isfinite(out[0, 1]).all()


def test_optional_outputs():
    t = _inputs((2, 3, 600), "f32", True)
    ref = msel.msel_lru_fwd(**t)
    out, final, chunks = msel.msel_lru_fwd(**t, return_final_state=False)
    assert final is None and chunks is None and torch.equal(out, ref[0])
    dout = normal((2, 3, 600), "f32", 6)
    g = msel.msel_lru_bwd(**t, dout=dout, want_dlam=False)
    assert g["dlam"] is None and g["dh0"] is None
    assert torch.equal(g["dx"], msel.msel_lru_bwd(**t, dout=dout)["dx"])


@pytest.mark.parametrize("shape", [(3, 50, 1), (3, 50, 7), (2, 9, 99), (2, 9, 300), (1, 5, 1500)])
def test_chunk_states_stand_for_the_carried_state(shape):
    """The backward starts from the chunk states that it is given, at every length: h0 itself is
    not needed then."""
    t = _inputs(shape, "f32", True)
    dout = normal(shape, "f32", 6)
    _, _, chunks = msel.msel_lru_fwd(**t, return_chunk_states=True)
    both = msel.msel_lru_bwd(**t, dout=dout, chunk_states=chunks, want_dh0=True)
    t["h0"] = None
    alone = msel.msel_lru_bwd(**t, dout=dout, chunk_states=chunks, want_dh0=True)
    for k in both:
        assert torch.equal(both[k], alone[k]), k


@pytest.mark.parametrize("shape", [(1, 130, 4700), (2, 100, 8300)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_blocks_of_a_row(shape, dtype):
    """Rows that a whole block of 16 wavefronts (8 in the backward) works on, over several of its
    tiles and a part of one."""
    log(f"lru blocks {shape} {dtype}")
    t = _inputs(shape, dtype, True)
    dout, dfinal = normal(shape, dtype, 6), normal(shape[:2], "f32", 7)
    out, final, chunks = msel.msel_lru_fwd(**t, return_chunk_states=True)
    ref = block.lru_fwd(*_oracle_args(t), values(t["h0"]))
    within("out", out, ref["out"], ref["out_err"])
    within("final", final, ref["final"], ref["final_err"])
    got = msel.msel_lru_bwd(**t, dout=dout, dfinal_state=dfinal, chunk_states=chunks,
                            want_dh0=True)
    ref = block.lru_bwd(*_oracle_args(t), values(dout), values(t["h0"]), values(dfinal))
    for k, r in (("dx", "dx"), ("dgate_a", "dga"), ("dgate_x", "dgx"), ("dlam", "dlam"),
                 ("dh0", "dh0")):
        within(k, got[k], ref[r], ref[r + "_err"])


@pytest.mark.parametrize("carried", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(5, 70, 14), (3, 41, 25), (7, 50, 32), (3, 70, 33), (2, 50, 50),
                                   (3, 37, 64), (2, 9, 65), (9, 31, 17)])
def test_short_rows(shape, dtype, carried):
    """Rows that 4, 8 or 16 lanes hold, in part and whole, with teams left over in the last block."""
    test_forward(shape, dtype, carried)
    test_backward(shape, dtype, carried)
