"""The oracle of the Muon step against what it has to do."""

import numpy as np
import pytest

from oracle import muon


@pytest.mark.parametrize("shape", [(4, 4), (8, 100), (100, 8), (1, 7), (7, 1)])
def test_singular_values_follow_the_polynomial(shape):
    """X keeps the singular vectors, and each singular value runs through the
    polynomial a s + b s^3 + c s^5."""
    rng = np.random.default_rng(shape[0])
    u = rng.standard_normal(shape)
    left, s, right = np.linalg.svd(u, full_matrices=False)
    s = s / (np.linalg.norm(u) + 1e-7)
    a, b, c = muon.COEFFICIENTS
    for _ in range(muon.STEPS):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(muon.orthogonalised(u), left * s @ right, atol=1e-9)
    # what the steps are for: values between about 0.7 and 1.2
    assert (s > 0.6).all() and (s < 1.3).all()


def test_transpose_and_scale_do_not_matter():
    u = np.random.default_rng(1).standard_normal((5, 40))
    x = muon.orthogonalised(u)
    assert np.allclose(muon.orthogonalised(u.T), x.T, atol=1e-12)
    assert np.allclose(muon.orthogonalised(1e6 * u, eps=1e-30), muon.orthogonalised(u, eps=1e-30),
                       atol=1e-9)
    assert (muon.orthogonalised(np.zeros((3, 9))) == 0).all()


def test_polynomial_of_the_gram_matrix_is_the_same():
    """The form that the library computes: T X0 with T a product of a I + b S + c
    S^2."""
    u = np.random.default_rng(2).standard_normal((6, 50))
    x = u / (np.linalg.norm(u) + 1e-7)
    s, t = x @ x.T, np.eye(6)
    a, b, c = muon.COEFFICIENTS
    for _ in range(muon.STEPS):
        q = a * np.eye(6) + b * s + c * s @ s
        s, t = s @ q @ q, t @ q
    assert np.allclose(t @ x, muon.orthogonalised(u), atol=1e-10)


def test_step_moves_against_the_gradient_and_decays():
    rng = np.random.default_rng(3)
    p, g = rng.standard_normal((4, 30)), rng.standard_normal((4, 30))
    m = np.zeros_like(p)
    p1, m1 = muon.step(p, g, m, 0.1, 0.9, True, 0.0)
    assert np.sum((p1 - p) * g) < 0
    assert np.allclose(m1, (1 - np.float64(np.float32(0.9))) * g)
    p2, _ = muon.step(p, 0 * g, m, 0.1, 0.9, False, 0.5)
    assert np.allclose(p2, p * (1 - np.float64(np.float32(0.1)) * 0.5))
    assert muon.factor("original", 400, 4) == 10 and muon.factor("original", 4, 400) == 1
    assert muon.factor("match_rms_adamw", 4, 100) == 2
