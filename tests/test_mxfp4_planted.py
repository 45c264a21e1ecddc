"""What the GPU comparisons of the MXFP4 product would notice (no GPU): mistakes planted in the oracle's operands."""
import numpy as np
import pytest

import gen
import oracle
from test_gpu_mxfp4 import random_held

M, N, K = 24, 40, 3300                                       # 26 groups of 128 columns, the last short


def operands(low, high):
    r = gen.rng(0, gen.KIND_MISC, 720, low)
    return random_held(r, M, K, low, high), random_held(r, N, K, low, high)


@pytest.mark.parametrize("places", [3, 4])
def test_stale_scales_are_noticed(places):
    """Scales in LDS go through `places` chunks of four groups.  A chunk that still held an earlier one's scales changes
    entries of the exact product, the first one that could (chunk `places`) as well as the last, short one."""
    a, b = operands(125, 127)
    want = oracle.mxfp4_matmul(a, b, K)
    for chunk in (places, (26 - 1) // 4):
        stale = b[1].copy()
        first, last = chunk * 16, min(chunk * 16 + 16, b[1].shape[1])
        stale[:, first:last] = b[1][:, first - places * 16:last - places * 16]
        assert np.mean(oracle.mxfp4_matmul(a, (b[0], stale), K) != want) > 0.9


def test_dropped_small_terms_are_noticed():
    """At the least scale: a product that takes all terms, or the terms below 2^-126, as zero."""
    a, b = operands(127, 127)
    a[1][:, : -(-K // 32)] = 0
    want = oracle.mxfp4_matmul(a, b, K)
    va, vb = oracle.mxfp4_values(*a, K), oracle.mxfp4_values(*b, K)
    terms = va[:, None, :] * vb[None, :, :]
    flushed = np.where(np.abs(terms) < 2.0 ** -126, 0.0, terms).sum(2)
    assert np.mean(want != 0) > 0.9 and np.mean(flushed != want) > 0.9
