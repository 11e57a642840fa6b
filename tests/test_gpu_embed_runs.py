"""The embedding's gradient where few ids hold long runs of tokens and the rows do not cancel: the
run's partial sums are added one after another, and their errors with them.

Bound: a chunk adds at most 32 rows in fp32 (31 u of its sum, all terms having one sign), the
partial sums are added in fp64, and the sum is rounded, scaled and rounded again: 40 u of the sum
of the terms' magnitudes covers it at any number of tokens."""
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402

from lm_helpers import U32  # noqa: E402


@pytest.mark.parametrize("tokens,dim", [(1 << 18, 256), (1 << 20, 40), ((1 << 20) + 5, 3)])
@pytest.mark.parametrize("kind", ["equal", "uniform"])
def test_one_id_for_every_token(tokens, dim, kind):
    log(f"embed one id {tokens}x{dim} {kind}")
    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    if kind == "equal":  # every token's row the same: rounding errors of one sign in a column
        dout = torch.empty(1, dim, device="cuda").uniform_(0.5, 1.5, generator=g)
        dout = dout.expand(tokens, dim).contiguous()
    else:
        dout = torch.empty(tokens, dim, device="cuda").uniform_(0.5, 1.5, generator=g)
    ids = torch.full((tokens,), 2, device="cuda")
    got = msel.msel_embed_bwd(ids, dout, 5, 0.5)
    ref = 0.5 * dout.double().sum(0)
    off = float(((got[2].double() - ref).abs() / (U32 * ref)).max())
    assert off <= 40.0, f"{off:.0f} u"
    assert not got[[0, 1, 3, 4]].any()
    assert torch.equal(got, msel.msel_embed_bwd(ids, dout, 5, 0.5))


def test_two_ids_onto_a_base():
    """Long runs of a few ids among short ones, added in place."""
    log("embed runs onto a base")
    tokens, dim, vocab = 1 << 19, 24, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(vocab, (tokens,), device="cuda", generator=g)
    ids[: tokens // 2] = 7
    ids[tokens // 2: tokens - 4096] = 250
    dout = torch.empty(tokens, dim, device="cuda").uniform_(0.5, 1.5, generator=g)
    base = torch.empty(vocab, dim, device="cuda").uniform_(0.5, 1.5, generator=g)
    ref = base.double().index_add(0, ids, dout.double())
    got = msel.msel_embed_bwd(ids, dout, vocab, base=base, dweight=base)
    off = float(((got.double() - ref).abs() / (U32 * ref)).max())
    assert off <= 40.0, f"{off:.0f} u"
