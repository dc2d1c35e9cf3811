"""Pins of the oracle's norm and orthogonalisation: hand-worked values, differences, singular values."""
import numpy as np
import pytest

from oracle import norm as ON
from oracle import ortho as OO

COEFFS = (3.4445, -4.7750, 2.0315)


def test_norm_of_a_hand_worked_row():
    h, rstd, y = ON.forward(np.array([[1.0, -3.0]]), np.array([[2.0, -1.0]]), np.array([1.0, 0.5]), 0.0)
    assert h.tolist() == [[3.0, -4.0]]
    np.testing.assert_allclose(rstd, [1 / np.sqrt(12.5)], rtol=1e-15)
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), -2 / np.sqrt(12.5)]], rtol=1e-15)


def test_scales_of_ragged_groups_and_zeros():
    y = np.zeros((2, 70))
    y[0, 3], y[0, 40], y[0, 69] = -448.0, 4.48, 0.0
    s = ON.scales(y, 32)
    assert s.shape == (2, 3)
    np.testing.assert_allclose(s[0], [1.0, 0.01, ON.SCALE_MIN])
    assert (s[1] == ON.SCALE_MIN).all()
    assert ON.spread(s, 32, 70).shape == (2, 70)
    assert ON.scales(y, 0).shape == (2, 1)


def test_backward_is_the_forward_s_difference_quotient():
    rng = np.random.default_rng(5)
    x, w, dy, dres = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))

    def loss(x, w):
        h, _, y = ON.forward(x, None, w, 1e-5)
        return (dy * y).sum() + (dres * h).sum()

    h, rstd, _ = ON.forward(x, None, w, 1e-5)
    dx, dw = ON.backward(dy, h, w, rstd, dres)
    e = 1e-6                                     # central differences: error e^2 and 2^-52 / e
    for i in np.ndindex(3, 7):
        d = np.zeros_like(x)
        d[i] = e
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * e) - dx[i]) < 1e-7
    for c in range(7):
        d = np.zeros_like(w)
        d[c] = e
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * e) - dw[c]) < 1e-7


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (6, 6), (1, 5), (1, 1)])
def test_orthogonalize_maps_singular_values_and_keeps_vectors(shape):
    u = np.random.default_rng(sum(shape)).normal(size=shape)
    left, s, right = np.linalg.svd(u, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    for _ in range(5):
        s = COEFFS[0] * s + COEFFS[1] * s ** 3 + COEFFS[2] * s ** 5
    got = OO.orthogonalize(u, 5, [COEFFS] * 5, 1e-7, scale=0.5)
    np.testing.assert_allclose(got, 0.5 * (left * s) @ right, atol=1e-11)


def test_momentum_step():
    g, m = np.array([[2.0]]), np.array([[10.0]])
    assert OO.momentum_step(g, m, 0.5, False)[0] == 7.0
    assert OO.momentum_step(g, m, 0.5, True)[0] == 5.5
    assert OO.momentum_step(g, m, 0.5, True)[1] == 7.0
