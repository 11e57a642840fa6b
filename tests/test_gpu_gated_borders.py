"""The gated norm at the widths where a block's passes end: groups one channel below and above what
it holds in registers and LDS, in tiles of 64 bytes (256 channels a pass, 12 passes held forward and
6 backward) and of 32 (512 channels a pass), with and without rows turned."""
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from lm_gpu_ref import check_backward, check_forward  # noqa: E402

# tokens: tiles of 64 bytes enough for these tiles, too few for tiles of 128; and tiles of 32
L64, L32 = {"bf16": 5201, "f32": 2601}, {"bf16": 1001, "f32": 501}


@pytest.mark.parametrize("n,length", [
    (1535, L64), (1537, L64), (3071, L64), (3073, L64), (3071, L32), (3073, L32), (6143, L32),
    (6145, L32)], ids=lambda v: str(v if isinstance(v, int) else v["bf16"]))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("first", [True, False])
def test_borders(n, length, dtype, first):
    log(f"gated borders {n} {length[dtype]} {dtype} {first}")
    case = (1, 1, n, length[dtype], dtype)
    for bld in (False, True):
        check_forward(case, first, bld)
        check_backward(case, first, bld)
