"""Pins of the 4-bit oracle: worked groups, rounding of the scale, ties of the codes."""
import numpy as np

from oracle import int4 as Q


def codes_of(c):
    return np.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)


def test_symmetric_group():
    w = np.zeros((1, 32))
    w[0, :8] = [7, -7, 0.5, 1.5, 2.5, -0.5, -1.5, 3.49]  # scale 1: ties go to even
    c, s, z = Q.quantize(w, 32, True)
    assert z is None and s[0, 0] == 1
    np.testing.assert_array_equal(codes_of(c)[0, :9], [15, 1, 8, 10, 10, 8, 6, 11, 8])
    np.testing.assert_array_equal(Q.values(c, s)[0, :9], [7, -7, 0, 2, 2, 0, -2, 3, 0])


def test_zero_point_group():
    w = np.zeros((1, 64))
    w[0, :4] = [-5, 10, 3, -2.5]
    w[0, 32:34] = [30, 15]
    c, s, z = Q.quantize(w, 32, False)
    np.testing.assert_array_equal(s, [[1, 2]])
    np.testing.assert_array_equal(z, [[5, 0]])
    np.testing.assert_array_equal(codes_of(c)[0, :5], [0, 15, 8, 3, 5])  # -2.5 rounds to -2
    np.testing.assert_array_equal(codes_of(c)[0, 32:35], [15, 8, 0])     # 7.5 rounds to 8


def test_scale_is_bf16():
    w = np.zeros((1, 32))
    w[0, 0] = 7 * (1 + 2.0 ** -8 + 2.0 ** -20)  # just above half a step of bf16 over 1
    assert Q.quantize(w, 32, True)[1][0, 0] == np.float32(1 + 2.0 ** -7)
    assert Q.bf16(np.float64(1 + 2.0 ** -8)) == 1 and Q.bf16(np.float64(1 + 3 * 2.0 ** -8)) == np.float32(1 + 2.0 ** -6)


def test_empty_and_nonfinite_groups():
    w = np.zeros((1, 96))
    w[0, 40], w[0, 70] = np.nan, 1e-39
    c, s, z = Q.quantize(w, 32, False)
    assert s[0, 0] == 1 and np.isnan(s[0, 1]) and s[0, 2] == 1
    np.testing.assert_array_equal(Q.values(c, s, z)[0, :32], 0)
    np.testing.assert_array_equal(Q.values(c, s, z)[0, 64:], 0)


def test_linear():
    rng = np.random.default_rng(0)
    c, s, z = Q.quantize(rng.standard_normal((5, 64)), 32, False)
    x, b = rng.standard_normal((3, 64)), rng.standard_normal(5)
    y, bound = Q.linear(x, c, s, z, b)
    np.testing.assert_allclose(y, x @ Q.values(c, s, z).T + b, rtol=1e-12)
    assert (bound > 0).all() and (bound < 1e-2).all()
