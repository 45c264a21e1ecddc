"""The MXFP4 kernels that the library holds (no GPU): every instance can be launched, every one that is launched is there.

The instances' names are read from the library that was built here."""
import os
import re

import pytest

from test_abi import gcl  # noqa: F401


@pytest.fixture(scope="module")
def names(gcl):  # noqa: F811
    with open(gcl.lib._name, "rb") as f:
        return f.read()


def test_decode_instances(names):
    """bf16, add, one long row, entries a thread: four entries are 16 bytes of float32, and half of a bf16 access."""
    got = set(re.findall(rb"mxfp4_decodeILb([01])ELb([01])ELb([01])ELi(\d+)E", names))
    flags = [(a, f) for a in (b"0", b"1") for f in (b"0", b"1")]
    assert got == {(b"0", a, f, n) for a, f in flags for n in (b"4", b"8")} | {(b"1", a, f, b"8") for a, f in flags}


def test_lds_waits_count_no_instructions():
    """A wait for LDS reads that leaves some of them out would rely on how many instructions the compiler makes of the
    reads behind it.  The sources wait for all, or use the values and leave the counting to the compiler."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gradient_compression_error_amd", "csrc")
    waits = []
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            waits += re.findall(r"lgkmcnt\(([^)]*)\)", f.read())
    assert set(waits) == {"0"}
