"""Log probabilities: rows that are not finite and rows that a mask leaves little of, in every kernel
that a row can be worked on by, beside rows that they must not reach."""
import math

import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402
from oracle import block  # noqa: E402

from block_helpers import normal, values, within  # noqa: E402

# (rows, vocab, top): teams of 4, 16 and 64 lanes, a block for a narrow row, rows held in registers,
# slices (held and not), whole wide rows with and without likeliest tokens
ROWS = [(5, 13, 5), (6, 60, 3), (7, 300, 8), (1030, 220, 20), (9, 1900, 4), (30, 250, 40),
        (600, 3001, 0), (4, 50257, 20), (3, 50257, 0), (2, 400001, 64), (520, 9001, 0), (520, 9001, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ROWS)
def test_rows_that_are_not_finite(shape, dtype):
    """A NaN or +inf makes the row's values and its whole gradient NaN, masked columns too, whatever is
    asked for with it, and leaves the other rows as they are, bit for bit."""
    log(f"logprob rows not finite {shape} {dtype}")
    rows, vocab, top = shape
    x = normal((rows, vocab), dtype, 1, 3.0)
    x[:, 1::5] = -math.inf
    ids = torch.zeros(rows, dtype=torch.int64, device="cuda")
    dlp, dh = normal((rows,), "f32", 2), normal((rows,), "f32", 3)

    def run(t):
        r = msel.msel_logprob_fwd(t, ids, 0.9, top, want_entropy=True)
        r["plain"] = msel.msel_logprob_fwd(t, ids, 0.9, top)["logprob"]
        r["dlogits"] = msel.msel_logprob_bwd(t, ids, r["lse"], dlp, dlp, dh, r["entropy"], 0.9)
        keep = t.clone()
        r["in_place"] = msel.msel_logprob_bwd(keep, ids, r["lse"], dlp, dlp, dh, r["entropy"], 0.9,
                                              dlogits=keep)
        return {k: v for k, v in r.items() if v is not None}
    clean = run(x)
    for bad in (math.nan, math.inf):
        for row in (0, rows - 1):
            for col in (2, vocab - 1):
                y = x.clone()
                y[row, col] = bad
                r = run(y)
                others = torch.arange(rows, device="cuda") != row
                for k, v in r.items():
                    assert torch.equal(v[others], clean[k][others]), k
                    if k == "top_ids":
                        assert int(v[row, 0]) == col and bool(((v >= 0) & (v < vocab)).all())
                        assert len(set(v[row].tolist())) == top
                    else:
                        assert bool(torch.isnan(v[row]).all()), (k, bad, row, col)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [20, 64])
@pytest.mark.parametrize("vocab", [250, 1900, 9001, 50257, 400001])
def test_few_tokens_that_are_allowed(vocab, top, dtype):
    """Rows of which a mask leaves no token, one, some dozens in one place, some dozens anywhere, and all
    but some dozens: the likeliest are those, then the masked ones from the first on, and the gradient
    stays on those that are left."""
    log(f"logprob few allowed {vocab} {top} {dtype}")
    x = torch.full((5, vocab), -math.inf, device="cuda", dtype=normal((1,), dtype).dtype)
    v = normal((5, vocab), dtype, 1, 3.0)
    some = torch.randperm(vocab, generator=torch.Generator().manual_seed(1))[:40].cuda()
    x[1, vocab // 3] = v[1, vocab // 3]
    x[2, vocab // 2:vocab // 2 + 40] = v[2, vocab // 2:vocab // 2 + 40]
    x[3, some] = v[3, some]
    x[4] = v[4]
    x[4, some] = -math.inf
    ids = torch.tensor([0, vocab // 3, vocab // 2, int(some[0]), int(some[0])], device="cuda")
    r = msel.msel_logprob_fwd(x, ids, 1.0, top, want_entropy=True)
    ref = block.logprob_fwd(values(x), ids.cpu().numpy(), 1.0, top)
    assert r["top_ids"].cpu().numpy().tolist() == ref["top_ids"].tolist()
    assert float(r["lse"][0]) == -math.inf and float(r["entropy"][0]) == 0.0
    one = torch.ones(5, device="cuda")
    d = msel.msel_logprob_bwd(x, ids, r["lse"], one)
    want, err = block.logprob_bwd(values(x), ids.cpu().numpy(), 1.0, values(one))
    within("dlogits", d[:4], want[:4], err[:4])
    # row 4's id is masked: its log probability is -inf, its gradient that of the formula
    assert float(r["logprob"][4]) == -math.inf
    within("dlogits", d[4], want[4], err[4])
