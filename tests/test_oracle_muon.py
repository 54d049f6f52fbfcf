"""Pins of the orthogonalisation oracle: singular vectors are kept and singular
values follow the scalar polynomial; tall is wide transposed; the cubic
coefficients converge to the polar factor; scale drops out; hand-checked step."""
import numpy as np
import pytest

from oracle import muon


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (6, 6), (1, 5), (5, 1)])
def test_singular_values_follow_the_scalar_steps(shape):
    x = np.random.default_rng(0).standard_normal(shape)
    u, s, vt = np.linalg.svd(x, full_matrices=False)
    t = s / np.sqrt((s * s).sum())
    a, b, c = muon.COEFFICIENTS
    for _ in range(5):
        t = a * t + b * t ** 3 + c * t ** 5
    assert np.allclose(muon.orthogonalize(x), (u * t) @ vt, atol=1e-12)
    assert np.all((t > 0.5) & (t < 1.3))


def test_transposed_and_scaled():
    x = np.random.default_rng(1).standard_normal((3, 7))
    assert np.allclose(muon.orthogonalize(x.T), muon.orthogonalize(x).T, atol=1e-14)
    assert np.allclose(muon.orthogonalize(1e6 * x), muon.orthogonalize(x), atol=1e-13)
    assert not muon.orthogonalize(0 * x).any()


def test_cubic_steps_reach_the_polar_factor():
    x = np.random.default_rng(2).standard_normal((4, 6))
    u, _, vt = np.linalg.svd(x, full_matrices=False)
    assert np.allclose(muon.orthogonalize(x, 40, (1.5, -0.5, 0.0)), u @ vt, atol=1e-12)


def test_step_of_a_single_value():
    # 1 x 1: X_0 = sign, five scalar steps
    t = 1.0
    a, b, c = muon.COEFFICIENTS
    for _ in range(5):
        t = a * t + b * t ** 3 + c * t ** 5
    p, m = muon.step([[2.0]], [[-3.0]], [[1.0]], lr=0.1, momentum=0.5, nesterov=False,
                     weight_decay=0.2, adjust=None)
    assert m[0, 0] == -1.0 and np.isclose(p[0, 0], 2.0 * 0.98 + 0.1 * t)
    p, m = muon.step([[2.0]], [[-3.0]], [[1.0]], lr=0.1, momentum=0.5, adjust="rms")
    assert np.isclose(p[0, 0], 2.0 + 0.02 * t)          # u = -2
    assert muon.factor("shape", 9, 4) == 1.5 and muon.factor("shape", 4, 9) == 1.0
