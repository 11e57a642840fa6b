"""The operators around the scan in the checked build: no kernel index leaves its buffer over a
range of shapes, and the outputs equal the release build's bit for bit."""
import numpy as np
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402
from selective_state_space_26_amd import _lib  # noqa: E402

from lm_helpers import normal  # noqa: E402


def _norm(rows, dim, dtype, rdtype):
    x, r = normal((rows, dim), dtype, 1), normal((rows, dim), rdtype, 2)
    w, dout = normal((dim,), "f32", 3), normal((rows, dim), dtype, 4)

    def run():
        out, s = msel.msel_norm_fwd(x, w, r)
        return [out, s, *msel.msel_norm_bwd(s, w, dout, r).values()]
    return run


def _gated(bsz, dim, L, groups, dtype, first, layout, out_layout):
    at = (bsz, dim, L) if layout == "bdl" else (bsz, L, dim)
    to = (bsz, dim, L) if out_layout == "bdl" else (bsz, L, dim)
    x, z, dout = normal(at, dtype, 1), normal(at, dtype, 2), normal(to, dtype, 3)
    w = normal((dim,), "f32", 4)
    a = (1e-5, groups, first, layout, out_layout)

    def run():
        return [msel.msel_gated_norm_fwd(x, z, w, *a),
                *msel.msel_gated_norm_bwd(x, z, w, dout, *a).values()]
    return run


def _embed(tokens, vocab, dim, dtype):
    r = np.random.default_rng([tokens, vocab])
    ids = torch.from_numpy(r.integers(-1, vocab + 1, tokens)).cuda()
    w, dout = normal((vocab, dim), "f32", 1), normal((tokens, dim), dtype, 2)

    def run():
        return [msel.msel_embed_fwd(ids, w, 2.0, dout.dtype),
                msel.msel_embed_bwd(ids, dout, vocab, 2.0, base=w)]
    return run


def _clip(sizes, dtype):
    t = [normal(s, dtype, i) for i, s in enumerate(sizes)]

    def run():
        out = [torch.zeros_like(x) for x in t]
        return [msel.msel_grad_clip(t, 0.5, out=out), *out]
    return run


CASES = {
    "norm_1": lambda: _norm(1, 1, "f32", "f32"),
    "norm_odd": lambda: _norm(37, 1027, "bf16", "f32"),
    "norm_wide": lambda: _norm(5, 16384, "bf16", "bf16"),
    "norm_rows": lambda: _norm(9000, 130, "f32", "f32"),
    "gated_rows": lambda: _gated(3, 300, 50, 3, "bf16", True, "bld", "bld"),
    "gated_short": lambda: _gated(4, 70, 3, 1, "f32", False, "bdl", "bld"),
    "gated_odd": lambda: _gated(2, 1537, 77, 1, "bf16", True, "bdl", "bld"),
    "gated_groups": lambda: _gated(1, 1000, 133, 4, "f32", False, "bdl", "bdl"),
    "gated_wide": lambda: _gated(1, 5121, 65, 1, "bf16", True, "bdl", "bld"),
    "gated_half_tiles": lambda: _gated(3, 1030, 700, 1, "bf16", True, "bdl", "bld"),
    "gated_half_tiles_f32": lambda: _gated(40, 1201, 21, 1, "f32", False, "bdl", "bdl"),
    "gated_small_blocks": lambda: _gated(300, 300, 19, 1, "bf16", True, "bdl", "bld"),
    "norm_narrow": lambda: _norm(5000, 20, "bf16", "bf16"),
    "embed_self_count": lambda: _embed(5000, 3000, 24, "bf16"),
    "embed_many_blocks": lambda: _embed(270000, 16, 8, "f32"),
    "gated_narrow_wide_tiles": lambda: _gated(3, 40, 5000, 1, "bf16", True, "bdl", "bld"),
    "gated_wide_tiles": lambda: _gated(1, 1601, 14500, 1, "bf16", True, "bdl", "bld"),
    "gated_wide_tiles_groups": lambda: _gated(2, 2400, 1000, 8, "f32", False, "bdl", "bdl"),
    "gated_widest": lambda: _gated(1, 16384, 40, 1, "f32", True, "bdl", "bdl"),
    "embed_small": lambda: _embed(5, 3, 2, "f32"),
    "embed_odd": lambda: _embed(3001, 777, 33, "bf16"),
    "embed_passes": lambda: _embed(40000, 300001, 5, "f32"),
    "embed_wide": lambda: _embed(600, 50, 2500, "bf16"),
    "clip": lambda: _clip([(1,), (4097,), (63, 63), (20000,)] + [(5, 3)] * 300, "bf16"),
}


@pytest.mark.parametrize("name", CASES)
def test_in_range_and_equal_to_release(name):
    log(f"checked build, {name}")
    run = CASES[name]()
    ref = [t.clone() for t in run()]
    with _lib.using(_lib.LIB_CHECKED_PATH):
        msel.bound_violations()
        got = run()
        count, f, line = msel.bound_violations()
        assert count == 0, f"{count} out-of-range indexes, the first at {f}:{line}"
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


WORKSPACES = {
    "gated": lambda b, d, L, g, t, w: msel.msel_gated_norm_bwd(
        *(normal((b, d, L), t, i) for i in (1, 2)), None, normal((b, L, d), t, 3), 1e-5, g, True,
        "bdl", "bld", workspace=w),
    "norm": lambda b, d, L, g, t, w: msel.msel_norm_bwd(
        normal((b * L, d), "f32", 1), None, normal((b * L, d), t, 2), workspace=w),
    "embed": lambda b, d, L, g, t, w: msel.msel_embed_bwd(
        torch.arange(b * L, device="cuda") % (b + g), normal((b * L, d), t, 2), b + g, workspace=w),
}
# few and many tiles of every width, short sequences, narrow and wide groups
SIZES = [(3, 1030, 700, 1), (40, 600, 40, 1), (30, 1030, 40, 2), (60, 520, 9, 1), (1, 1536, 300, 1),
         (2, 700, 3, 1), (600, 24, 17, 2), (9, 2000, 130, 4), (5, 520, 1500, 1), (230, 70, 64, 1)]


@pytest.mark.parametrize("op", list(WORKSPACES))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_is_written_behind_the_workspace(op, dtype):
    guard = 1 << 20
    for size in SIZES:
        log(f"workspace {op} {dtype} {size}")
        asked = []

        def ask(workspace, need, dev):
            asked.append(need)
            buf = torch.full((need + guard,), 0x5A, device=dev, dtype=torch.uint8)
            asked.append(buf)
            return buf, need  # the library is told of the size that it asked for

        with pytest.MonkeyPatch.context() as m:
            for mod in ("norm", "embed"):
                m.setattr(f"selective_state_space_26_amd.{mod}._workspace", ask)
            WORKSPACES[op](*size, dtype, None)
        torch.cuda.synchronize()
        need, buf = asked
        assert need > 0 and bool((buf[need:] == 0x5A).all()), size
