"""The MXFP4 oracle (CPU): hand-worked blocks, the rounding borders, and invariants of the step with memory."""
import numpy as np
import pytest

import gen
import oracle


def codes_of(row):
    c, s = oracle.mxfp4_quantize(np.asarray([row], np.float32))
    flat = np.stack([c[0] & 15, c[0] >> 4], 1).ravel()
    return flat[: len(row)].tolist(), s[0].tolist()


def test_hand_block():
    # largest 6.0: E = 129, s = 127, scale 1: the E2M1 magnitudes are their own codes
    row = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.5, -6.0]
    c, s = codes_of(row)
    assert c == [0, 1, 2, 3, 4, 5, 6, 7, 9, 15]
    assert s == [127, 0, 0, 0]
    # the same block times 2^-9: only the scale moves
    c2, s2 = codes_of([v * 2.0 ** -9 for v in row])
    assert c2 == c and s2 == [118, 0, 0, 0]


def test_rounding_borders_and_saturation():
    # scale 1 (largest 7.75 in [4, 8)); ties go to the even code, above 6 saturates
    up = lambda v: float(np.nextafter(np.float32(v), np.float32(9)))       # noqa: E731
    down = lambda v: float(np.nextafter(np.float32(v), np.float32(0)))     # noqa: E731
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    row = [7.75] + [f(b) for b in borders for f in (down, lambda v: v, up)]
    c, s = codes_of(row)
    assert s[0] == 127 and c[0] == 7
    want = []
    for i, _ in enumerate(borders):
        want += [i, i if i % 2 == 0 else i + 1, i + 1]
    assert c[1:] == want


def test_scale_range():
    # 2^127 (largest exponent), the least normal, subnormals, zeros
    assert codes_of([3.0e38])[1][0] == 252
    assert codes_of([2.0 ** -126])[1][0] == 0
    assert codes_of([2.0 ** -130])[0] == [0] and codes_of([2.0 ** -130])[1][0] == 0     # 2^-130 / 2^-127 = 0.125
    assert codes_of([2.0 ** -128])[0] == [1]
    assert codes_of([0.0, -0.0]) == ([0, 8], [0, 0, 0, 0])


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_not_finite(bad):
    x = np.ones((1, 70), np.float32)
    x[0, 40] = bad
    c, s = oracle.mxfp4_quantize(x)
    assert s[0].tolist() == [125, 255, 125, 0] and np.all(c[0, 16:32] == 0)
    v = oracle.mxfp4_values(c, s, 70)[0]
    assert np.isnan(v[32:64]).all() and np.array_equal(v[:32], np.ones(32)) and np.array_equal(v[64:], np.ones(6))


def test_nearest_by_brute_force():
    r = gen.rng(0, gen.KIND_MISC, 300)
    x = r.standard_normal((7, 200), dtype=np.float32) * np.exp(r.uniform(-20, 20, (7, 1))).astype(np.float32)
    c, s = oracle.mxfp4_quantize(x)
    v = oracle.mxfp4_values(c, s, 200)
    grid = np.concatenate([-np.array([6, 4, 3, 2, 1.5, 1, 0.5]), [0, 0.5, 1, 1.5, 2, 3, 4, 6]])
    for i in range(7):
        for j in range(200):
            g = grid * 2.0 ** (int(s[i, j // 32]) - 127)
            assert abs(v[i, j] - np.float64(x[i, j])) == np.abs(g - np.float64(x[i, j])).min()
    # the largest of every block lies in [4, 8) of its scale
    top = np.abs(np.pad(x, ((0, 0), (0, 56))).reshape(7, -1, 32)).max(2)[:, :6]
    ratio = top / np.ldexp(1.0, s[:, :6].astype(int) - 127)
    assert np.all((ratio >= 4) & (ratio < 8))


def test_step_invariants():
    """m' + g = acc up to the one rounding of m'; the step contracts: what is left is at most a third of each block's
    largest entry (a border at 5 between 4 and 6, or 8 - 6 above it, over at least 4)."""
    mem, eta = gen.gaussian_vector(1000, 7, 0.1), 0.3
    g = gen.gaussian_vector(1000, 8)
    r = oracle.mxfp4_ef_step(mem, g, eta)
    left = r["acc"].astype(np.float64) - r["g"]
    assert np.array_equal(r["mem"], left.astype(np.float32))
    top = np.abs(np.pad(r["acc"], (0, 24)).reshape(-1, 32)).max(1)
    assert np.all(np.abs(np.pad(left, (0, 24)).reshape(-1, 32)).max(1) <= top / 3)
    # with the memory, what was sent adds up to what came in
    total, sent, mem = np.zeros(1000), np.zeros(1000), np.zeros(1000, np.float32)
    for t in range(50):
        g = gen.gaussian_vector(1000, 100 + t)
        r = oracle.mxfp4_ef_step(mem, g, 1.0)
        total, sent, mem = total + g, sent + r["g"], r["mem"]
    # 50 steps of two roundings of values below 16
    assert np.abs(total - sent - mem).max() <= 100 * 8 * 2.0 ** -24
