"""Calls of the MXFP4 binding that need no GPU: what it has to refuse before the C call sees it."""
import pytest
import torch

from test_abi import gcl  # noqa: F401


@pytest.mark.parametrize("count", [2**20 + 1, 2**31, 2**32 + 1])
def test_more_messages_than_an_int_holds(gcl, count):  # noqa: F811
    """One stored message seen as many: 2^32 + 1 of them would reach the C call as one."""
    codes = torch.zeros(64, dtype=torch.uint8).expand(count, 64)
    scales = torch.zeros(4, dtype=torch.uint8).expand(count, 4)
    with pytest.raises(ValueError, match="2\\^20 messages"):
        gcl.gc_mxfp4_decode(codes, scales, torch.zeros(5))
