"""Pins of the oracle's layer norm, expert rows and AdamW: hand-worked values, differences, statistics."""
import numpy as np

from oracle import adamw as OA
from oracle import experts as OE
from oracle import norm as ON


def test_layer_norm_of_a_hand_worked_row():
    h, mean, rstd, y = ON.layer_forward(np.array([[1.0, 2.0]]), np.array([[2.0, 5.0]]), np.array([1.0, 0.5]), np.array([0.0, 3.0]), 0.0)
    assert h.tolist() == [[3.0, 7.0]] and mean.tolist() == [5.0] and rstd.tolist() == [0.5]
    assert y.tolist() == [[-1.0, 3.5]]


def test_layer_norm_s_backward_is_the_forward_s_difference_quotient():
    rng = np.random.default_rng(6)
    x, dy, dres = (rng.normal(size=(3, 7)) for _ in range(3))
    w, b = rng.normal(size=7), rng.normal(size=7)

    def loss(x, w, b):
        h, _, _, y = ON.layer_forward(x, None, w, b, 1e-5)
        return (dy * y).sum() + (dres * h).sum()

    h, mean, rstd, _ = ON.layer_forward(x, None, w, b, 1e-5)
    grads = dict(zip("xwb", ON.layer_backward(dy, h, w, mean, rstd, dres)))
    e = 1e-6
    for name in "xwb":
        args = {"x": x, "w": w, "b": b}
        for i in np.ndindex(*args[name].shape):
            d = np.zeros_like(args[name])
            d[i] = e
            up, down = (loss(**{**args, name: args[name] + s * d}) for s in (1, -1))
            assert abs((up - down) / (2 * e) - grads[name][i]) < 1e-7


def test_route_of_a_hand_worked_batch():
    ids = np.array([[3, 1], [1, 9], [-1, 3], [3, 3]])
    position, offsets, counts = OE.route(ids, experts=3, first=1, align=4, max_rows=100)
    assert position.tolist() == [[4, 0], [1, -1], [-1, 5], [6, 7]]
    assert offsets.tolist() == [0, 4, 4, 8] and counts.tolist() == [2, 0, 4]
    assert OE.filled(offsets, counts) == [2, 3]
    position, offsets, counts = OE.route(ids, experts=3, first=1, align=4, max_rows=6)
    assert position.tolist() == [[4, 0], [1, -1], [-1, 5], [-1, -1]]
    assert offsets.tolist() == [0, 4, 4, 6] and counts.tolist() == [2, 0, 2]


def test_combine_and_its_gradients_are_each_other_s_differences():
    rng = np.random.default_rng(7)
    position = np.array([[2, 0], [-1, 1], [-1, -1]])
    rows, weights, dout = rng.normal(size=(4, 5)), rng.normal(size=(3, 2)), rng.normal(size=(3, 5))
    loss = lambda r, w: (OE.combine(r, position, w)[0] * dout).sum()  # noqa: E731
    drows, dweights, _ = OE.combine_backward(dout, rows, position, weights, np.array([0, 3]), np.array([3]), np.zeros((4, 5)))
    for i in np.ndindex(4, 5):                   # linear in each: differences are exact but for rounding
        d = np.zeros((4, 5))
        d[i] = 1.0
        assert abs(loss(rows + d, weights) - loss(rows, weights) - drows[i]) < 1e-12
    for i in np.ndindex(3, 2):
        d = np.zeros((3, 2))
        d[i] = 1.0
        assert abs(loss(rows, weights + d) - loss(rows, weights) - dweights[i]) < 1e-12


def test_adamw_s_first_step_is_the_sign_times_the_rate():
    g = np.array([2.0, -1e-3, 5.0])
    p, m, v = OA.step(np.array([1.0, 1.0, 0.0]), g, np.zeros(3), np.zeros(3), 1, 0.1, (0.9, 0.999), 1e-12, 0.5)
    np.testing.assert_allclose(p, [0.95 - 0.1, 0.95 + 0.1, -0.1], rtol=1e-8)
    np.testing.assert_allclose(m, 0.1 * g)
    np.testing.assert_allclose(v, 0.001 * g * g)
    half = OA.step(np.ones(3), g, np.zeros(3), np.zeros(3), 1, 0.1, (0.9, 0.999), 1e-12, 0.0, grad_scale=0.5)
    np.testing.assert_allclose(half[1], 0.05 * g)


def test_the_random_bits_are_spread_evenly_and_independently():
    """Counts of 16 equal classes of each kind over 2^18 elements: 2^14 expected, standard deviation 124; of the three kinds'
    256 pairs of classes 2^10 expected, 32.  Six of them allowed (a chance of 2e-9 a class)."""
    n = 1 << 18
    kinds = [b >> 12 for b in OA.noise(123, 7, 5, np.arange(n))]
    for b in kinds:
        assert np.abs(np.bincount(b, minlength=16) - n / 16).max() < 6 * 124
    for a, b in ((0, 1), (0, 2), (1, 2)):
        assert np.abs(np.bincount(kinds[a] * 16 + kinds[b], minlength=256) - n / 256).max() < 6 * 32
    # neighbours, another step, another tensor, another seed, and the same place 2^32 elements on
    for other in (OA.noise(123, 7, 5, np.arange(n) + 1), OA.noise(123, 8, 5, np.arange(n)), OA.noise(123, 7, 6, np.arange(n)),
                  OA.noise(124, 7, 5, np.arange(n)), OA.noise(123, 7, 5, np.arange(n) + 2 ** 32)):
        for k in range(3):
            assert np.abs(np.bincount(kinds[k] * 16 + (other[k] >> 12), minlength=256) - n / 256).max() < 6 * 32


def test_stochastic_rounding_keeps_values_on_the_grid_and_the_mean():
    for x, step in ((1.3, 0.125), (-300.0, 32.0), (0.011, 2.0 ** -9), (0.0, 2.0 ** -9)):
        got = OA.stochastic(np.full(65536, x), np.arange(65536), 4, 2.0 ** -6)
        assert set(np.unique(got / step) % 1) == {0.0} and abs(got.mean() - x) <= step / 65536
    assert OA.spacing(np.array([2.0 ** -6, 2.0 ** -7, 448.0]), 4, 2.0 ** -6).tolist() == [2.0 ** -9, 2.0 ** -9, 32.0]


def test_scales_of_a_ragged_tensor():
    x = np.zeros(130)
    x[3], x[129] = -44.8, 448.0
    np.testing.assert_allclose(OA.scales(x), [0.1, 1.0])
    assert OA.spread(OA.scales(x), 130).shape == (130,)
