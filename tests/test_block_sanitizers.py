"""The host code of the gated recurrence, the log probabilities and the feed-forward block (argument
checks, plans and workspace sizing, the entry points' early returns) under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU, as test_lm_sanitizers.py does for the operators around the
scan: the GPU code is built as usual and never launched."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import CSRC, HIPCC, ROOT, SAN_HOST, SOURCES, _run

# row_norm.hip has the sums of partial rows that the recurrence's backward ends with
BLOCK_SOURCES = ["block_api.cpp", "lru.hip", "logprob.hip", "gated_mlp.hip", "row_norm.hip"]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_host_code_under_asan_ubsan(tmp_path):
    inc = os.path.join(ROOT, "include")

    def compile_one(src):
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        _run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
              *SAN_HOST, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-munsafe-fp-atomics", "-I", inc, "-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    sources = BLOCK_SOURCES + SOURCES  # msel_api.cpp has the shared entry points
    with ThreadPoolExecutor(max_workers=8) as ex:
        objs = list(ex.map(compile_one, sources))
    drv = str(tmp_path / "block_driver.o")
    _run([HIPCC, "-x", "c", "-O1", "-g", *SAN_HOST, "-I", inc, "-c",
          os.path.join(ROOT, "tests", "sanitize", "block_driver.c"), "-o", drv])
    exe = str(tmp_path / "block_driver")
    _run([HIPCC, "--offload-arch=gfx950", *SAN_HOST, "-o", exe, drv, *objs, "-L/opt/rocm/lib",
          "-lamdhip64"])
    # the HIP runtime keeps allocations until exit by design: leak reports are not ours
    r = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert "all checks passed" in r.stdout
