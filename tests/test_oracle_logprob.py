"""Pins of the log-probability oracle: worked rows, masks, and its gradient against differences."""
import numpy as np

from oracle import logprob as L


def test_worked_rows():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.2, 0.7, 0.1]])) + 3.0
    lp, h, tl, ti = L.token_logprobs(x, np.array([1, -100]), 2)
    np.testing.assert_allclose(lp, [np.log(0.25), 0.0], rtol=1e-12)
    np.testing.assert_allclose(h, [1.5 * np.log(2), -(0.2 * np.log(0.2) + 0.7 * np.log(0.7) + 0.1 * np.log(0.1))], rtol=1e-12)
    np.testing.assert_array_equal(ti, [[0, 1], [1, 0]])  # the tie goes to 1
    np.testing.assert_allclose(tl, np.log([[0.5, 0.25], [0.7, 0.2]]), rtol=1e-12)


def test_masks():
    x = np.array([[-np.inf, 0.0, -np.inf], [-np.inf] * 3])
    lp, h, tl, ti = L.token_logprobs(x, np.array([0, 1]), 2)
    np.testing.assert_array_equal(lp, [-np.inf, -np.inf])
    np.testing.assert_array_equal(h, [0, 0])
    np.testing.assert_array_equal(ti, [[1, -1], [-1, -1]])
    np.testing.assert_array_equal(tl, [[0, -np.inf], [-np.inf, -np.inf]])
    np.testing.assert_array_equal(L.gradient(np.ones(2), np.ones(2), x, np.array([0, 1])), [[0, -1, 0], [0, 0, 0]])


def test_gradient_by_differences():
    rng = np.random.default_rng(0)
    x, t = rng.standard_normal((4, 7)) * 2, np.array([3, 0, -1, 6])
    g, h = rng.standard_normal(4), rng.standard_normal(4)
    d = L.gradient(g, h, x, t)

    def f(v):
        lp, e, _, _ = L.token_logprobs(v, t)
        return (g * lp).sum() + (h * e).sum()
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-5
        # third derivatives below 10, times step^2 / 6; 2^-52 of a sum of about 20 over the step
        assert abs((f(x + e) - f(x - e)) / 2e-5 - d[i]) <= 10 * 1e-10 / 6 + 20 * 2.0 ** -52 / 1e-5
