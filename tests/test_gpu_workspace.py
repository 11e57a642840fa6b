"""A caller's workspace for the scan's backwards: taken when it is large enough, and refused when
it is not contiguous memory of the GPU (here pinned host memory, which a kernel could reach)."""
import pytest

import msel_inputs
from helpers import log, to_device

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import selective_state_space_26_amd as msel  # noqa: E402

BSZ, DIM, N, L = 2, 8, 16, 600


def _call(op, workspace):
    d = to_device(msel_inputs.make(BSZ, DIM, N, L, "f32", 77, with_dout=True))
    a = (d["A"], d["B"], d["C"], d["dout"])
    if op == "scan":
        return msel.msel_scan_bwd(d["u"], d["delta"], *a, workspace=workspace)
    if op == "trap":
        lam = torch.full_like(d["u"], 0.5)
        return msel.msel_scan_trap_bwd(d["u"], d["delta"], lam, *a, workspace=workspace)
    return msel.msel_scan_complex_bwd(d["u"], d["delta"], *a, workspace=workspace)


@pytest.mark.parametrize("op", ["scan", "trap", "complex"])
def test_given_workspaces(op):
    log(f"workspace {op}")
    size = 1 << 24
    for bad in (torch.empty(size, dtype=torch.uint8, pin_memory=True),
                torch.empty(size // 1024, 1024, device="cuda", dtype=torch.uint8).t()):
        with pytest.raises(ValueError):
            _call(op, bad)
    with pytest.raises(TypeError):
        _call(op, 12345)
    ref = _call(op, None)
    got = _call(op, torch.full((size,), 0x7F, device="cuda", dtype=torch.uint8))
    for k in ("du", "ddelta"):
        assert torch.equal(ref[k], got[k]), k
