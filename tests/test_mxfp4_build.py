"""The MXFP4 kernels that the library holds (no GPU): every instance can be launched, every one that is launched is there.

The instances' names are read from the library that was built here."""
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
