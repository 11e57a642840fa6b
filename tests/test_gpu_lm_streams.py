"""The operators around the scan run on the stream that is current: their inputs are written on a
side stream behind long work there, so that a call that went to another stream would read what was
in them before."""
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402

from lm_helpers import normal  # noqa: E402


def _inputs():
    return {
        "x": normal((2, 300, 1000), "bf16", 1), "z": normal((2, 300, 1000), "bf16", 2),
        "dout": normal((2, 1000, 300), "bf16", 3), "w": normal((300,), "f32", 4),
        "rows": normal((500, 300), "bf16", 5), "res": normal((500, 300), "f32", 6),
        "ids": torch.arange(3000, device="cuda") % 70, "table": normal((70, 300), "f32", 7),
        "drow": normal((3000, 300), "bf16", 8), "g0": normal((300, 400), "f32", 9),
        "g1": normal((77,), "bf16", 10),
    }


def _clip(t):
    out = [torch.full_like(g, float("nan")) for g in (t["g0"], t["g1"])]
    return [msel.msel_grad_clip([t["g0"], t["g1"]], 0.5, out=out), *out]


CALLS = {
    "norm_fwd": lambda t: list(msel.msel_norm_fwd(t["rows"], t["w"], t["res"])),
    "norm_bwd": lambda t: list(msel.msel_norm_bwd(t["res"], t["w"], t["rows"],
                                                  t["res"]).values()),
    "gated_fwd": lambda t: [msel.msel_gated_norm_fwd(t["x"], t["z"], t["w"], out_layout="bld")],
    "gated_bwd": lambda t: list(msel.msel_gated_norm_bwd(t["x"], t["z"], t["w"], t["dout"],
                                                         out_layout="bld").values()),
    "embed_fwd": lambda t: [msel.msel_embed_fwd(t["ids"], t["table"], 2.0)],
    "embed_bwd": lambda t: [msel.msel_embed_bwd(t["ids"], t["drow"], 70, 2.0)],
    "clip": _clip,
    "grad_norm": lambda t: [msel.msel_grad_norm([t["g0"], t["g1"]])],
}


@pytest.mark.parametrize("op", CALLS)
def test_runs_on_the_current_stream(op):
    log(f"streams {op}")
    t = _inputs()
    ref = CALLS[op](t)
    keep = {k: v.clone() for k, v in t.items()}
    for v in t.values():
        v.zero_()
    m = torch.randn(4096, 4096, device="cuda").bfloat16()
    out = torch.empty_like(m)
    torch.mm(m, m, out=out)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(200):  # some 100 us each
            torch.mm(m, m, out=out)
        for k, v in t.items():
            v.copy_(keep[k])
        got = [r.clone() for r in CALLS[op](t)]
        for v in t.values():  # and a call that came later would read zeros
            v.zero_()
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
