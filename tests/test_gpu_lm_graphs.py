"""The operators around the scan only enqueue kernels on the caller's stream (no memset, no
allocation inside the library, no synchronisation): their steps are captured in a HIP graph and
replayed.  Every replay, after its outputs were overwritten, its inputs changed in place and the
eager step run between, must match the eager step bit for bit: all of them are deterministic."""
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402

from lm_helpers import normal  # noqa: E402


def _norm():
    x, r, w = normal((97, 515), "bf16", 1), normal((97, 515), "f32", 2), normal((515,), "f32", 3)

    def step():
        out, s = msel.msel_norm_fwd(x, w, r)
        return dict(out=out, s=s, **msel.msel_norm_bwd(s, w, out, s))
    return step, [x, r, w]


def _gated(layout, L):
    def make():
        shape = (2, 96, L) if layout == "bdl" else (2, L, 96)
        x, z, w = normal(shape, "bf16", 1), normal(shape, "bf16", 2), normal((96,), "f32", 3)

        def step():
            out = msel.msel_gated_norm_fwd(x, z, w, layout=layout, out_layout="bld")
            return dict(out=out, **msel.msel_gated_norm_bwd(x, z, w, out, layout=layout,
                                                           out_layout="bld"))
        return step, [x, z, w]
    return make


def _embed(tokens):
    def make():
        w = normal((700, 72), "f32", 1)
        ids = torch.randint(-1, 701, (tokens,), generator=torch.Generator().manual_seed(2)).cuda()

        def step():
            out = msel.msel_embed_fwd(ids, w, 2.0, torch.bfloat16)
            return dict(out=out, dweight=msel.msel_embed_bwd(ids, out, 700, 2.0, base=w))
        return step, [w, ids]
    return make


def _clip():
    ts = [normal((n,), ("f32", "bf16")[i % 2], i) for i, n in enumerate([5, 70000, 1, 3001])]

    def step():
        outs = [torch.empty_like(t) for t in ts]
        norm = msel.msel_grad_clip(ts, 1.5, out=outs)
        return dict(norm=norm, **{f"t{i}": o for i, o in enumerate(outs)})
    return step, ts


STEPS = {"norm": _norm, "gated": _gated("bdl", 1500), "gated_short": _gated("bdl", 3),
         "gated_one": _gated("bdl", 1), "gated_rows": _gated("bld", 70), "embed": _embed(9000),
         "embed_few": _embed(300), "clip": _clip}


@pytest.mark.parametrize("name", list(STEPS))
def test_replays_match_eager_steps(name):
    log(f"graph {name}")
    step, inputs = STEPS[name]()
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()  # warm up on the capture stream
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            cap = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for k in range(4):
        for t in inputs:  # new values in the same memory
            t.copy_(t.flip(0) if not t.is_floating_point() else t.flip(0) * 0.75)
        for t in cap.values():
            t.fill_(float("nan"))
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(cap[n], eager[n]), (k, n)
