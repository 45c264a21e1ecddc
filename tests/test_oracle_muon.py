"""The oracle of the orthogonalised update (CPU): singular values, invariants, hand-worked cases."""
import numpy as np
import pytest

import gen
import oracle


def quintic(s, steps, coefs=(3.4445, -4.7750, 2.0315)):
    a, b, c = (float(np.float32(v)) for v in coefs)
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return s


@pytest.mark.parametrize("n,m", [(1, 1), (1, 9), (9, 1), (8, 8), (6, 20), (20, 6)])
def test_acts_on_singular_values(n, m):
    """The step keeps singular vectors and maps each singular value by the quintic."""
    u = gen.rng(0, gen.KIND_MISC, 1000, n * 100 + m).standard_normal((n, m))
    left, s, right = np.linalg.svd(u, full_matrices=False)
    for steps in (1, 2, 5):
        want = (left * quintic(s / np.sqrt(np.sum(s * s)), steps)) @ right
        assert np.allclose(oracle.newton_schulz(u, steps), want, atol=1e-12)


def test_drives_singular_values_towards_one():
    u = gen.rng(0, gen.KIND_MISC, 1001).standard_normal((40, 70))
    s = np.linalg.svd(oracle.newton_schulz(u), compute_uv=False)
    assert 0.65 < s.min() and s.max() < 1.25


def test_other_coefficients_converge():
    """The cubic 1.5 s - 0.5 s^3 over many steps gives the polar factor."""
    u = gen.rng(0, gen.KIND_MISC, 1002).standard_normal((5, 8))
    left, _, right = np.linalg.svd(u, full_matrices=False)
    assert np.allclose(oracle.newton_schulz(u, 32, (1.5, -0.5, 0.0)), left @ right, atol=1e-10)
    per_step = [(1.0, 0.0, 0.0), (2.0, 0.0, 0.0)]
    assert np.allclose(oracle.newton_schulz(u, 2, per_step), 2 * u / np.linalg.norm(u))


def test_momentum():
    g = np.array([[1.0, 2.0]], np.float32)
    m = np.array([[10.0, -4.0]], np.float32)
    got = oracle.muon_step(g, m, 0.5, True)
    assert np.array_equal(got["mem"], [[6.0, 0.0]]) and np.array_equal(got["u"], [[4.0, 2.0]])
    got = oracle.muon_step(g, m, 0.5, False, scale=3.0)
    assert np.array_equal(got["u"], [[6.0, 0.0]])
    assert np.allclose(got["out"], [[3 * quintic(1.0, 5), 0.0]])
    assert oracle.muon_step(g, None, 0.5, True)["mem"] is None


def test_zero_and_not_finite():
    assert np.array_equal(oracle.newton_schulz(np.zeros((3, 4))), np.zeros((3, 4)))
    x = np.ones((3, 4))
    for bad in (np.nan, np.inf, -np.inf):
        x[1, 2] = bad
        assert np.isnan(oracle.newton_schulz(x)).all()
