"""The embedding lookup and its gradient on the GPU against the fp64 oracle: table and
activation dtypes, both id types, widths around the vectors and teams, vocabularies of one and
more sort passes, one token, runs that cross segment chunks, one id for every token, ids outside
the table, a padding id, a base gradient beside and in place.  Bounds: lm_helpers."""
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


def _ids(tokens, vocab, kind, seed=0, dtype=torch.int64):
    r = np.random.default_rng([seed, tokens, vocab])
    if kind == "uniform":
        a = r.integers(0, vocab, tokens)
    elif kind == "zipf":
        a = np.minimum(np.floor(np.exp(r.random(tokens) * np.log(vocab + 1.0)) - 1.0), vocab - 1)
    elif kind == "one":
        a = np.full(tokens, vocab // 2)
    else:  # "outside": some ids that no table row has
        a = r.integers(-3, vocab + 4, tokens)
        a[::7] = vocab
        a[3::11] = -1
    return torch.from_numpy(a.astype(np.int64)).to(dtype).cuda()


@pytest.mark.parametrize("dim", [1, 4, 7, 8, 33, 64, 768, 1027, 2500])
@pytest.mark.parametrize("wdtype", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_fwd(dim, wdtype, dtype):
    log(f"embed fwd {dim} {wdtype} {dtype}")
    w = normal((97, dim), wdtype, 1)
    for idt in (torch.int64, torch.int32):
        ids = _ids(3 * 41, 97, "outside", 1, idt).reshape(3, 41)
        out = msel.msel_embed_fwd(ids, w, 3.5, DTYPES[dtype])
        assert tuple(out.shape) == (3, 41, dim)
        # one product and one rounding
        assert_elementwise("out", out, lm.embed_fwd(ids.cpu().numpy(), host(w), 3.5), k=1.0)


def test_embed_fwd_one_token_is_a_row():
    log("embed fwd one token")
    w = normal((1000, 768), "f32", 1)
    out = msel.msel_embed_fwd(torch.tensor([[999]], device="cuda"), w)
    assert torch.equal(out[0, 0], w[999])


BWD = [
    # tokens, vocab, dim, ids
    (1, 1, 1, "uniform"), (1, 50, 8, "uniform"), (31, 7, 5, "uniform"), (32, 3, 64, "uniform"),
    (33, 1, 9, "one"), (1000, 16, 64, "uniform"), (1024, 511, 40, "zipf"),
    (1025, 512, 33, "uniform"), (3000, 2000, 96, "outside"), (5000, 70000, 24, "zipf"),
    (40000, 11, 16, "uniform"), (9000, 300000, 3, "zipf"), (4096, 100, 768, "one"),
    (2048, 50, 1030, "zipf"), (8192, 50, 16, "zipf"), (8193, 900, 12, "outside"),
    (700, 40, 2500, "outside"), (140000, 3000, 4, "zipf"),
]


@pytest.mark.parametrize("case", BWD, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_bwd(case, dtype):
    tokens, vocab, dim, kind = case
    log(f"embed bwd {case} {dtype}")
    ids = _ids(tokens, vocab, kind, 3, torch.int32 if tokens % 2 else torch.int64)
    dout = normal((tokens, dim), dtype, 4)
    dw = msel.msel_embed_bwd(ids, dout, vocab, 2.0)
    ref, terms = lm.embed_bwd(ids.cpu().numpy(), host(dout), vocab, 2.0)
    assert_sum("dweight", dw, ref, terms)
    again = msel.msel_embed_bwd(ids, dout, vocab, 2.0)
    assert torch.equal(dw, again)  # a fixed order of additions


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_embed_bwd_base_and_padding(dtype):
    log(f"embed bwd base {dtype}")
    tokens, vocab, dim = 2500, 300, 50
    ids = _ids(tokens, vocab, "zipf", 5).reshape(50, 50)
    dout, base = normal((50, 50, dim), dtype, 6), normal((vocab, dim), "f32", 7)
    ref, terms = lm.embed_bwd(ids.cpu().numpy(), host(dout), vocab, 0.5, host(base), padding_idx=0)
    dw = msel.msel_embed_bwd(ids, dout, vocab, 0.5, base=base, padding_idx=0)
    assert_sum("dweight", dw, ref, terms)
    assert torch.equal(dw[0], base[0])
    keep = base.clone()
    got = msel.msel_embed_bwd(ids, dout, vocab, 0.5, base=keep, padding_idx=0, dweight=keep)
    assert got is keep and torch.equal(got, dw)


def test_embed_bwd_without_any_valid_token():
    log("embed bwd all ids outside")
    ids = torch.full((100,), -1, device="cuda")
    dw = msel.msel_embed_bwd(ids, normal((100, 12), "f32", 1), 5)
    assert not dw.any()


def test_embed_bwd_nonfinite_rows_stay_in_their_row():
    log("embed bwd non-finite")
    ids = torch.arange(200, device="cuda") % 20
    dout = normal((200, 12), "f32", 1)
    dout[47] = float("nan")  # token 47 is id 7
    dw = msel.msel_embed_bwd(ids, dout, 20)
    bad = torch.isnan(dw).any(1)
    assert bad[7] and int(bad.sum()) == 1


@pytest.mark.parametrize("bad", ["ids", "cpu", "table", "dout", "base", "vocab"])
def test_embed_refusals(bad):
    ids, w = torch.zeros(4, dtype=torch.int64, device="cuda"), normal((5, 8), "f32", 1)
    dout = normal((4, 8), "f32", 2)
    with pytest.raises((TypeError, ValueError, _lib.MselError)):
        if bad == "ids":
            msel.msel_embed_fwd(ids.float(), w)
        elif bad == "cpu":
            msel.msel_embed_fwd(ids.cpu(), w)
        elif bad == "table":
            msel.msel_embed_fwd(ids, w.t())
        elif bad == "dout":
            msel.msel_embed_bwd(ids, dout[:3], 5)
        elif bad == "base":
            msel.msel_embed_bwd(ids, dout, 5, base=w.bfloat16())
        else:
            msel.msel_embed_bwd(ids, dout, 0)
