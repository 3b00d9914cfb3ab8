"""Pins of the grouped router's oracle: worked rows, and its gradient against differences."""
import numpy as np
import pytest

from oracle import router as R
from oracle import serving as S


def test_worked_row():
    # scores 0.5 0.75 0.9 0.25 | 0.6 0.6 0.1 0.1 | 0.95 0 0 0; groups worth 1.65, 1.2, 0.95
    p = np.array([[0.5, 0.75, 0.9, 0.25, 0.6, 0.6, 0.1, 0.1, 0.95, 1e-9, 1e-9, 1e-9]])
    x = np.log(p / (1 - p))
    w, ids = R.group_gate(x, 3, groups=3, group_k=2, scale=2.0)
    np.testing.assert_array_equal(ids, [[2, 1, 4]])  # the tie of 4 and 5 goes to 4
    np.testing.assert_allclose(w, [2 * np.array([0.9, 0.75, 0.6]) / 2.25], rtol=1e-12)
    _, ids = R.group_gate(x, 3, groups=3, group_k=2, group_top=1)  # worth 0.9, 0.6, 0.95
    np.testing.assert_array_equal(ids, [[8, 2, 1]])
    bias = np.zeros(12)
    bias[6] = 1.0
    w, ids = R.group_gate(x, 2, bias=bias, renormalize=False)
    np.testing.assert_array_equal(ids, [[6, 8]])
    np.testing.assert_allclose(w, [[0.1, 0.95]], rtol=1e-12)  # the bias selects and does not weigh


def test_masked():
    x = np.full((2, 6), -np.inf)
    x[1, 4] = 0.0
    w, ids = R.group_gate(x, 2, groups=3, group_k=1)
    np.testing.assert_array_equal(ids, [[-1, -1], [4, -1]])
    np.testing.assert_array_equal(w, [[0, 0], [1, 0]])


def test_softmax_without_groups_is_the_plain_router():
    x = np.random.default_rng(0).standard_normal((20, 24)) * 3
    for renorm in (True, False):
        w, ids = R.group_gate(x, 5, score="softmax", renormalize=renorm)
        wo, io = S.moe_gate(x, 5, renorm)
        np.testing.assert_array_equal(ids, io)
        np.testing.assert_allclose(w, wo, rtol=1e-13)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_by_differences(score, renorm):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 12)) * 2
    _, ids = R.group_gate(x, 4, rng.standard_normal(12) * 0.1, 3, 2, 2, score, renorm, 1.5)
    g = rng.standard_normal((3, 4))
    d = R.group_gate_grad(g, ids, x, score, renorm, 1.5)
    f = lambda v: (g * R.fixed_weights(v, ids, score, renorm, 1.5)).sum()
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        # central differences: third derivatives (below 4) times step^2, and 2^-52 of a sum of about 5 over the step
        assert abs((f(x + e) - f(x - e)) / 2e-6 - d[i]) <= 1e-11 + 5 * 2.0 ** -52 / 1e-6 * 2
