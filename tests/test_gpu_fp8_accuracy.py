"""GPU: how far sums of the 8-bit matrix instructions (results in bf16) are off, and when.

They add eight products at a time, each cut off 13 places below the leading bit of the largest of the eight: less than
2^-13 of that one each, so a sum is off by less than 7 * 2^-13 times the sum of the magnitudes of its terms, however small
the sum itself is.  Beside it the float32 sum's own roundings, k 2^-23 of the sum of magnitudes.

What a bf16 result's own rounding hides is seen by adding the product to the negative of its rounded value: the difference
is small, so rounding it costs 2^-8 of it only."""
import numpy as np
import pytest
import torch

import gen
import oracle
from gpu_util import DEV, lib, require_gpu, to_dev
from test_gpu_fp8 import Held, product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def quantized(x):
    h = Held(*x.shape)
    lib().gc_fp8_quantize(to_dev(x), *h.pair)
    return h.host()


def off(a, b, m, n, k):
    """(the bf16 kernels' sums minus the exact ones, up to 2^-8 of the exact sums' own rounding; the exact sums)."""
    va, vb = (torch.from_numpy(oracle.fp8_values(*h, k)).to(DEV) for h in (a, b))
    want = va @ vb.t().contiguous()
    rounded = want.to(torch.bfloat16)
    got = product(a, b, m, n, k, dtype=torch.bfloat16, old=(-rounded).float().cpu().numpy()).to(DEV)
    return got.double() - (want - rounded.double()), want, va, vb


SHAPES = [(16, 1000, 4096), (247, 356, 993), (451, 365, 586), (1075, 979, 517), (763, 722, 1995), (385, 449, 7121), (1667, 2362, 940),
          (3970, 4000, 1500)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_normal_entries(m, n, k):
    """Normal entries: about 1.5e-5 of the results' size, as the header says (root of the mean squares).  Rounding to bf16 is off
    by 1.7e-3 of a result, rounding the difference by 1.7e-3 of that: 3e-6."""
    print(f"case: fp8 bf16 sums of normal entries {m}x{n}x{k}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 995, k)
    a, b = (quantized(r.standard_normal((rows, k), dtype=np.float32)) for rows in (m, n))
    e, want, _, _ = off(a, b, m, n, k)
    rms = float(e.square().mean().sqrt() / want.square().mean().sqrt())
    print(f"rms {rms:.3g}", flush=True)
    assert 0.7e-5 <= rms <= 2.1e-5                           # half as much again, or half


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_outliers_that_cancel(m, n, k):
    """Two products of 2^14 that cancel, beside others of about one: the sum is as large as without them, but what is added with
    them is cut to multiples of 2, so six to fourteen terms are lost: 2 to 4, of a sum of sqrt(k) (85 at most)."""
    print(f"case: fp8 bf16 sums with outliers {m}x{n}x{k}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 996, k)
    x, y = (r.standard_normal((rows, k), dtype=np.float32) for rows in (m, n))
    x[:, 3], x[:, 4] = 128, -128                             # (held exactly: the scale of their group is 2^-1)
    y[:, 3] = y[:, 4] = 128
    a, b = quantized(x), quantized(y)
    e, want, va, vb = off(a, b, m, n, k)
    rms = float(e.square().mean().sqrt() / want.square().mean().sqrt())
    size = va.abs() @ vb.abs().t().contiguous()
    bound = (1 + 2.0 ** -8) * (7 * 2.0 ** -13 + k * 2.0 ** -23) * size + 2.0 ** -16 * want.abs()
    print(f"rms {rms:.3g}, largest of the bound {float((e.abs() / bound).max()):.3g}", flush=True)
    assert bool((e.abs() <= bound).all()) and rms > 1e-3
    # the float32 result of the same operands: exact products, float32 sums
    got = product(a, b, m, n, k).double().to(DEV)
    assert bool(((got - want).abs() <= k * 2.0 ** -23 * size).all())
