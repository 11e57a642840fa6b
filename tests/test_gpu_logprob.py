"""Log probabilities of tokens on the GPU against their definition in fp64: narrow rows in
registers, wide rows, rows in slices, masks, ties, strided rows, gradients in place."""
import math

import numpy as np
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402
from oracle import block  # noqa: E402

from block_helpers import DTYPES, normal, values, within  # noqa: E402

# (rows, vocab): the borders of 4, 16 and 64 lanes per row in both types, blocks, slices
SHAPES = [(1, 1), (3, 2), (7, 3), (130, 16), (5, 63), (9, 64), (9, 65), (4, 128), (4, 129),
          (20, 257), (6, 513), (5, 1024), (5, 1025), (3, 2049), (700, 2500), (2, 4097),
          (2, 8200), (1, 50257), (37, 20011)]


def _ids(rows, vocab, seed=9):
    r = np.random.default_rng([seed, rows, vocab])
    ids = r.integers(0, vocab, rows)
    ids[::7] = (-100, vocab, -1)[seed % 3]
    return torch.from_numpy(ids).cuda()


def _check(r, ref, top):
    within("logprob", r["logprob"], ref["logprob"], ref["logprob_err"])
    within("lse", r["lse"], ref["lse"], ref["lse_err"])
    within("entropy", r["entropy"], ref["entropy"], ref["entropy_err"])
    if top:
        assert np.array_equal(r["top_ids"].cpu().numpy(), ref["top_ids"])
        within("top", r["top_logprobs"], ref["top_logprobs"], ref["top_err"])


@pytest.mark.parametrize("scale", [1.0, 0.6])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype, scale):
    log(f"logprob forward {shape} {dtype} {scale}")
    x, ids = normal(shape, dtype, 1, 3.0), _ids(*shape)
    top = min(shape[1], 64 if scale == 1.0 else 5)
    r = msel.msel_logprob_fwd(x, ids, scale, top, want_entropy=True)
    _check(r, block.logprob_fwd(values(x), ids.cpu().numpy(), scale, top), top)
    # each output is the same when it is asked for alone
    alone = msel.msel_logprob_fwd(x, ids.int(), scale)
    assert alone["entropy"] is None and alone["top_ids"] is None
    within("lse", alone["lse"], values(r["lse"]), np.abs(values(r["lse"])) * 4 + 32)
    none = msel.msel_logprob_fwd(x, scale=scale, top=top, want_lse=False)
    assert none["logprob"] is None and none["lse"] is None
    assert torch.equal(none["top_ids"], r["top_ids"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype):
    log(f"logprob backward {shape} {dtype}")
    x, ids = normal(shape, dtype, 1, 3.0), _ids(*shape, seed=10)
    dlp, dl, dh = (normal(shape[:1], "f32", s) for s in (2, 3, 4))
    for scale, a in ((1.0, dict(dlogprob=dlp)), (0.6, dict(dlogprob=dlp, dlse=dl, dentropy=dh)),
                     (1.7, dict(dentropy=dh))):
        f = msel.msel_logprob_fwd(x, ids, scale, want_entropy=True)
        ref, err = block.logprob_bwd(values(x), ids.cpu().numpy(), scale,
                                     *(values(a.get(k)) for k in ("dlogprob", "dlse", "dentropy")))
        entropy = f["entropy"] if "dentropy" in a else None
        d = msel.msel_logprob_bwd(x, ids, f["lse"], entropy=entropy, scale=scale, **a)
        within("dlogits", d, ref, err)
        keep = x.clone()
        same = msel.msel_logprob_bwd(keep, ids, f["lse"], entropy=entropy, scale=scale,
                                     dlogits=keep, **a)
        assert same is keep and torch.equal(keep, d)


MASKED = [(3, 5), (9, 16), (4, 100), (5, 700), (3, 3001), (3, 20011)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", MASKED)
def test_masked_rows(shape, dtype):
    """Columns of -inf, a row with one column left, one with none, and masks of the type's lowest
    value."""
    log(f"logprob masked {shape} {dtype}")
    x = normal(shape, dtype, 1, 3.0)
    x[torch.rand(shape, generator=torch.Generator().manual_seed(3)).cuda() < 0.6] = -math.inf
    x[0] = -math.inf
    x[1] = -math.inf
    x[1, shape[1] // 2] = 1.25
    low = torch.finfo(DTYPES[dtype]).min
    x[2] = torch.where(torch.isinf(x[2]), low, x[2])
    x[2, 0] = 0.5
    ids = _ids(*shape, seed=9)
    ids[0], ids[1], ids[2] = 0, shape[1] // 2, 0
    top = min(shape[1], 20)
    r = msel.msel_logprob_fwd(x, ids, 1.0, top, want_entropy=True)
    assert float(r["lse"][0]) == -math.inf and float(r["entropy"][0]) == 0.0
    assert float(r["logprob"][0]) == -math.inf and float(r["logprob"][1]) == 0.0
    v = values(x)
    _check(r, block.logprob_fwd(v, ids.cpu().numpy(), 1.0, top), top)
    dlp, dh = normal(shape[:1], "f32", 2), normal(shape[:1], "f32", 4)
    d = msel.msel_logprob_bwd(x, ids, r["lse"], dlp, None, dh, r["entropy"])
    ref, err = block.logprob_bwd(v, ids.cpu().numpy(), 1.0, values(dlp), None, values(dh))
    within("dlogits", d, ref, err)
    assert bool((d[0] == 0).all())


@pytest.mark.parametrize("vocab", [50, 700, 9000])
def test_rows_of_the_lowest_value(vocab):
    """All columns at the lowest value are alike: uniform."""
    log(f"logprob lowest {vocab}")
    x = torch.full((2, vocab), torch.finfo(torch.float32).min, device="cuda")
    ids = torch.tensor([0, vocab - 1], device="cuda")
    r = msel.msel_logprob_fwd(x, ids, want_entropy=True, top=1)
    # sums of ones are exact, the logarithm is off by 2 roundings
    within("logprob", r["logprob"], np.full(2, -np.log(vocab)), 4 * np.log(vocab))
    within("entropy", r["entropy"], np.full(2, np.log(vocab)), 4 * np.log(vocab))
    d = msel.msel_logprob_bwd(x, ids, r["lse"], torch.ones(2, device="cuda"))
    ref = np.full((2, vocab), -1.0 / vocab)
    ref[[0, 1], [0, vocab - 1]] += 1.0
    within("dlogits", d, ref, 16.0 / vocab + 2 * np.abs(ref))


@pytest.mark.parametrize("shape", [(3, 60), (3, 900), (2, 6001), (1, 40000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_go_to_the_lowest_id(shape, dtype):
    """Few distinct values (more ties than any list of candidates holds), zeros of both signs."""
    log(f"logprob ties {shape} {dtype}")
    g = torch.Generator().manual_seed(4)
    x = (torch.randint(-2, 2, shape, generator=g).to(DTYPES[dtype]) * 0.0
         + torch.randint(0, 2, shape, generator=g)).to(DTYPES[dtype]).cuda()
    x[0] = -0.0
    x[0, ::3] = 0.0
    for top in (1, 20, 60):
        r = msel.msel_logprob_fwd(x, top=top)
        ref = block.logprob_fwd(values(x), None, 1.0, top)
        assert np.array_equal(r["top_ids"].cpu().numpy(), ref["top_ids"]), top


@pytest.mark.parametrize("shape", [(2, 40), (3, 300), (2, 9000)])
def test_what_is_not_finite(shape):
    """NaN and +inf make their row NaN and leave the others; the ids stay in range."""
    log(f"logprob non-finite {shape}")
    x = normal(shape, "f32", 1)
    x[0, 7] = float("nan")
    x[1, 5] = math.inf
    ids = torch.zeros(shape[0], dtype=torch.int64, device="cuda")
    r = msel.msel_logprob_fwd(x, ids, top=8, want_entropy=True)
    for k in ("logprob", "lse", "entropy"):
        assert torch.isnan(r[k][:2]).all() or k == "lse" and math.isnan(float(r[k][0])), k
        assert torch.isfinite(r[k][2:]).all(), k
    assert int(r["top_ids"][0, 0]) == 7 and int(r["top_ids"][1, 0]) == 5
    assert bool(((r["top_ids"] >= 0) & (r["top_ids"] < shape[1])).all())
    x[0] = float("nan")
    assert r["top_ids"].shape == (shape[0], 8)
    assert msel.msel_logprob_fwd(x, top=8)["top_ids"][0].tolist() == list(range(8))


@pytest.mark.parametrize("vocab", [60, 1500, 5000])
def test_large_logits(vocab):
    """Logits around 1e5: an fp32 lse has too few digits, the gradient sums the row again."""
    log(f"logprob large {vocab}")
    x = normal((3, vocab), "f32", 1) + 1e5
    ids = torch.tensor([1, 2, 3], device="cuda")
    r = msel.msel_logprob_fwd(x, ids)
    one = torch.ones(3, device="cuda")
    shifted, err = block.logprob_bwd(values(x) - 1e5, ids.cpu().numpy(), 1.0, values(one))
    d = msel.msel_logprob_bwd(x, ids, r["lse"], one)
    within("dlogits", d, shifted, err)
    keep = x.clone()
    assert torch.equal(msel.msel_logprob_bwd(keep, ids, r["lse"], one, dlogits=keep), d)


@pytest.mark.parametrize("vocab,width,start", [(50, 64, 0), (1000, 1030, 3), (5000, 5004, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_rows(vocab, width, start, dtype):
    """The first columns of a padded vocabulary, and nothing is written beside them.  A row's vectors
    start with its line of memory, so rows at other addresses are summed in another order: both are
    within the bounds of the sums, which hold for any order.  The ids, and the gradient for the same
    sums, are equal."""
    log(f"logprob strided {vocab} {dtype}")
    wide = normal((2, 5, width), dtype, 1, 3.0)
    x = wide[..., start:start + vocab]
    ids = _ids(10, vocab).view(2, 5)
    dlp = normal((2, 5), "f32", 2)
    c = x.contiguous()
    a = msel.msel_logprob_fwd(x, ids, top=4, want_entropy=True)
    b = msel.msel_logprob_fwd(c, ids, top=4, want_entropy=True)
    ref = block.logprob_fwd(values(c), ids.cpu().numpy(), 1.0, 4)
    _check(a, ref, 4)
    _check(b, ref, 4)
    assert a["top_ids"].shape == (2, 5, 4)
    ref = msel.msel_logprob_bwd(c, ids, b["lse"], dlp)
    d = msel.msel_logprob_bwd(x, ids, b["lse"], dlp)
    assert d.is_contiguous() and torch.equal(d, ref)
    keep = wide.clone()
    at = keep[..., start:start + vocab]
    msel.msel_logprob_bwd(at, ids, b["lse"], dlp, dlogits=at)
    assert torch.equal(at, ref)
    at.copy_(x)
    assert torch.equal(keep, wide)


def test_refusals():
    x = normal((4, 100), "f32", 1)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    lse = torch.zeros(4, device="cuda")
    bad = [lambda: msel.msel_logprob_fwd(x, ids.float()), lambda: msel.msel_logprob_fwd(x, ids[:3]),
           lambda: msel.msel_logprob_fwd(x.t(), top=1), lambda: msel.msel_logprob_fwd(x.cpu()),
           lambda: msel.msel_logprob_fwd(x.half()), lambda: msel.msel_logprob_fwd(x, top=101),
           lambda: msel.msel_logprob_fwd(x, top=-1), lambda: msel.msel_logprob_fwd(x, top=65),
           lambda: msel.msel_logprob_fwd(x, ids, scale=0.0),
           lambda: msel.msel_logprob_fwd(x, ids, scale=math.inf),
           lambda: msel.msel_logprob_fwd(x, want_lse=False),
           lambda: msel.msel_logprob_fwd(x[:0]),
           lambda: msel.msel_logprob_bwd(x, ids, None, lse),
           lambda: msel.msel_logprob_bwd(x, None, lse, lse),
           lambda: msel.msel_logprob_bwd(x, ids, lse, dentropy=lse),
           lambda: msel.msel_logprob_bwd(x, ids, lse.double(), lse),
           lambda: msel.msel_logprob_bwd(x, ids, lse, lse, dlogits=x.bfloat16()),
           lambda: msel.msel_logprob_bwd(x[:, :50], ids, lse, lse, dlogits=x[:, 25:75]),
           lambda: msel.msel_logprob_bwd(x[:2], ids[:2], lse[:2], lse[:2], dlogits=x[1:3])]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            f()
            pytest.fail(f"call {i} was not refused")


@pytest.mark.parametrize("vocab", [50, 700, 1500, 9000, 40000])
@pytest.mark.parametrize("scale", [3.0e38, 1e-38])
def test_scales_at_the_ends_of_fp32(vocab, scale):
    """At the largest scale a row's largest logit has all the probability, at the smallest every
    logit the same."""
    x = normal((3, vocab), "f32", 3).clamp(-8, 8)
    ids = torch.tensor([0, 1, 2], device="cuda")
    best = torch.tensor([0, 9, 2], device="cuda")
    x.scatter_(1, best[:, None], 9.0)
    r = msel.msel_logprob_fwd(x, ids, scale, want_entropy=True)
    one, dh = torch.ones(3, device="cuda"), torch.full((3,), 0.5, device="cuda")
    d = msel.msel_logprob_bwd(x, ids, r["lse"], one, None, dh, r["entropy"], scale)
    if scale > 1:
        assert r["logprob"].tolist() == [0.0, -float("inf"), 0.0]
        assert r["entropy"].tolist() == [0.0, 0.0, 0.0]
        want = torch.zeros_like(x)
        want[1, 1], want[1, 9] = scale, -scale
        assert torch.equal(d, want)
    else:
        # log V and its negative to a few roundings of their sums (V / 256 + 20 terms one after another)
        lse = torch.log(torch.tensor(float(vocab), dtype=torch.float64))
        for k, v in (("logprob", -lse), ("lse", lse), ("entropy", lse)):
            assert (r[k].double().cpu() - v).abs().max() < 2 ** -24 * (vocab / 256 + 40 + 4 * lse)
        assert torch.isfinite(d).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 17), (5, 250), (900, 256), (1030, 200), (4, 500), (600, 897),
                                   (6, 1800), (1025, 1000)])
def test_many_likeliest_tokens_of_narrow_rows(shape, dtype):
    """Up to 64 tokens, where a block takes a narrow row for them and where teams do."""
    test_forward(shape, dtype, 1.0)
