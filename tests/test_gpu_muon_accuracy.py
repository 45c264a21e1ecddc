"""GPU: what gc_muon_step's results are accurate to, beyond the bounds of test_gpu_muon."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import require_gpu
from test_gpu_muon import USUAL, matrix, step

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


SETS = [[(1, 1), (33, 31)], [(64, 576)], [(100, 64)], [(130, 257), (300, 200), (257, 1000)], [(1024, 1024)], [(2048, 300)],
        [(2100, 2300)], [(4097, 4000)]]


@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("shapes", SETS, ids=lambda s: "+".join(f"{n}x{m}" for n, m in s))
def test_bf16_is_the_float32_result_rounded_once(shapes, steps):
    """Every step is the same for either type of out; the tiles of each product, odd and even groups of k."""
    print(f"case: muon bf16 against float32 {shapes} steps {steps}", flush=True)
    grads = [matrix(n, m, "low", 40) for n, m in shapes]
    exact, _ = step(grads, steps=steps)
    got, _ = step(grads, steps=steps, out_dtype=torch.bfloat16)
    for w, g in zip(exact, got):
        assert torch.equal(g, w.to(torch.bfloat16))


def least(x, b, c, dx, da, dp):
    """What held values' least value puts on one step's result, entry by entry: X off by dx, A by da and P by dp at most."""
    big = np.abs(x) @ np.abs(x).T
    p = b * big + c * (big @ big)
    off_a = dx * (np.abs(x).sum(1)[:, None] + np.abs(x).sum(1)[None, :]) + da
    off_p = b * off_a + c * (big @ off_a + off_a @ big) + dp
    return dx * p.sum(1, keepdims=True) + off_p @ np.abs(x), p


@pytest.mark.parametrize("down", [-12, -20, -24, -31, -36])
@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("n,m", [(64, 576), (576, 64), (33, 31), (130, 257), (300, 1111), (1500, 1400), (3010, 2990)])
def test_parts_much_smaller_than_the_rest(n, m, axis, down):
    """Half of the rows, or of the columns, `down` binades below the others: one step, entry by entry.  The bound is
    test_gpu_muon's with what the pairs cannot hold at the powers of two that a step of singular values up to 1 has: X and
    A 2^15 and P 2^14 times themselves, lo 2^11 times that but for the largest shape here, whose tiles are of 192: each off by
    half of f16's least value, 2^-25."""
    print(f"case: muon {n}x{m}, parts 2^{down} along {axis}", flush=True)
    low = 2.0 ** 11 if n < 2000 else 1.0
    u = matrix(n, m, "gauss", 41)
    small = np.exp2(down).astype(np.float32)
    (u if axis == 0 else u.T)[::2] *= small
    x = u.astype(np.float64) / np.linalg.norm(u.astype(np.float64))
    x = x.T if n > m else x
    k, w = x.shape
    a, b, c = (abs(float(np.float32(v))) for v in USUAL)
    floor, p = least(x, b, c, 2.0 ** -40 / low, 2.0 ** -40 / low, 2.0 ** -39 / low)
    e = 9 * 2.0 ** -22 + 3 * (w + 2 * k) * 2.0 ** -23
    d = 9 * 2.0 ** -22 + 3 * k * 2.0 ** -23
    bound = 2 * (e * (p @ np.abs(x)) + d * a * np.abs(x) + floor + a * 2.0 ** -40 / low)
    want = oracle.newton_schulz(u, 1)
    want = want.T if n > m else want
    (got,), _ = step([u], steps=1)
    got = got.double().numpy()
    assert np.all(np.abs((got.T if n > m else got) - want) <= bound)


@pytest.mark.parametrize("n,m", [(33, 50), (50, 33)])
def test_small_and_large_scales(n, m):
    """A scale is one rounding of each entry, 2^-24 of it, as far as the results are normal."""
    print(f"case: muon {n}x{m}, scales near float32's ends", flush=True)
    u = matrix(n, m, "gauss", 42)
    (one,), _ = step([u])
    one = one.double().numpy()
    for scale in (1.1e-36, -3.3e-33, 1.7e38):
        (got,), _ = step([u], scales=[scale])
        want = one * float(np.float32(scale))
        normal = np.abs(want) >= 2.0 ** -126
        assert normal.mean() > 0.5
        assert np.all(np.abs(got.double().numpy() - want)[normal] <= 2.0 ** -24 * np.abs(want)[normal])
