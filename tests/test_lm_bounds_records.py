"""Every source with kernels keeps a record of out-of-range indexes; the reader of the records
declares those of the operators around the scan weakly, so that a build of the scan alone links.
A library as it is shipped has all of them (CPU)."""
import ctypes
import os
import re

import pytest

from selective_state_space_26_amd import _lib, build
from selective_state_space_26_amd.scan import BOUNDS_FILES

HIP = sorted(f for f in os.listdir(build.CSRC) if f.endswith(".hip"))


def _taker(source):
    with open(os.path.join(build.CSRC, source)) as f:
        return re.search(r"^MSEL_BOUNDS_TAKER\((\w+)\)", f.read(), re.M).group(1)


def test_every_source_is_built_and_named():
    assert set(HIP) <= set(build.SOURCES)
    assert sorted(BOUNDS_FILES.values()) == HIP
    assert sorted(BOUNDS_FILES) == list(range(1, len(HIP) + 1))


@pytest.mark.parametrize("path", [_lib.LIB_PATH, _lib.LIB_CHECKED_PATH])
def test_the_library_has_every_record(path):
    lib = ctypes.CDLL(path)
    for source in HIP:
        name = _taker(source)
        assert hasattr(lib, f"_ZN4msel{len(name)}{name}EPNS_12BoundsRecordE"), source


def test_records_are_read_in_the_order_of_their_numbers():
    with open(os.path.join(build.CSRC, "msel_api.cpp")) as f:
        text = f.read()
    table = text[text.index("const Taker takers[]"):]
    listed = re.findall(r"msel::(take_bounds_\w+)", table[:table.index("};")])
    assert listed == [_taker(BOUNDS_FILES[i]) for i in sorted(BOUNDS_FILES)]
