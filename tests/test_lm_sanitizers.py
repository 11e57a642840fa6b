"""The host code of the operators around the scan (argument checks, workspace sizing, the entry
points' early returns) under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: the
sources are built with the sanitizers on the host side only (the GPU code is built as usual and
never launched) and driven by tests/sanitize/lm_driver.c, which exits 0 when its expectations
hold; a sanitizer finding aborts it."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import CSRC, HIPCC, ROOT, SAN_HOST, SOURCES, _run

LM_SOURCES = ["lm_api.cpp", "row_norm.hip", "tile_norm.hip", "tile_norm_bwd.hip",
              "tile_short.hip", "embed.hip", "grads.hip"]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_host_code_under_asan_ubsan(tmp_path):
    inc = os.path.join(ROOT, "include")

    def compile_one(src):
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        _run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
              *SAN_HOST, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-munsafe-fp-atomics", "-I", inc, "-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    sources = LM_SOURCES + SOURCES  # the bounds reports of msel_api.cpp reach all of them
    with ThreadPoolExecutor(max_workers=8) as ex:
        objs = list(ex.map(compile_one, sources))
    drv = str(tmp_path / "lm_driver.o")
    _run([HIPCC, "-x", "c", "-O1", "-g", *SAN_HOST, "-I", inc, "-c",
          os.path.join(ROOT, "tests", "sanitize", "lm_driver.c"), "-o", drv])
    exe = str(tmp_path / "lm_driver")
    _run([HIPCC, "--offload-arch=gfx950", *SAN_HOST, "-o", exe, drv, *objs, "-L/opt/rocm/lib",
          "-lamdhip64"])
    # the HIP runtime keeps allocations until exit by design: leak reports are not ours
    r = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert "all checks passed" in r.stdout
