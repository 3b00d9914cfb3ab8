"""Pins of the 64-bit oracle of the router, the few-token expert layer and the
8-bit products (no GPU)."""
import numpy as np
import pytest

from oracle import serving as S


def test_gate_worked_rows():
    inf = np.inf
    x = np.array([[1.0, 3.0, 3.0, 2.0], [-inf, -inf, 5.0, -inf], [-inf] * 4, [np.nan, 1.0, -inf, 0.0],
                  [-0.0, 0.0, -1.0, -2.0]])
    w, ids = S.moe_gate(x, 2)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [1, 3], [0, 1]]
    np.testing.assert_allclose(w[:2], [[0.5, 0.5], [1.0, 0.0]])
    np.testing.assert_array_equal(w[2], [0, 0])
    np.testing.assert_allclose(w[3], np.array([1, np.exp(-1)]) / (1 + np.exp(-1)))
    w, _ = S.moe_gate(x[:1], 2, renormalize=False)
    np.testing.assert_allclose(w[0], [1 / (2 + np.exp(-1) + np.exp(-2))] * 2)


def test_gate_weights_sum_and_order():
    x = np.random.default_rng(0).standard_normal((50, 30))
    w, ids = S.moe_gate(x, 7)
    np.testing.assert_allclose(w.sum(1), 1)
    assert (np.diff(w, axis=1) <= 0).all()
    assert all(len(set(r)) == 7 for r in ids.tolist())


@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(renorm):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((6, 12))
    x[2, :9] = -np.inf
    k = 5
    _, ids = S.moe_gate(x, k, renorm)
    g = rng.standard_normal((6, k))
    d = S.moe_gate_grad(g, ids, x, renorm)
    f = lambda z: (np.where(ids >= 0, g, 0) * S.fixed_weights(z, ids, renorm)).sum()
    h = 1e-5
    for t in range(6):
        for e in range(12):
            if not np.isfinite(x[t, e]):
                assert d[t, e] == 0
                continue
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((f(up) - f(dn)) / (2 * h) - d[t, e]) < 1e-9


def test_moe_few_is_the_sum_of_experts():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 16))
    w13, w2 = rng.standard_normal((4, 32, 16)), rng.standard_normal((4, 16, 16))
    ids = np.array([[0, 3], [-1, 2], [-1, -1]], dtype=np.int32)
    w = np.array([[0.25, 0.75], [9.0, 1.0], [1.0, 1.0]])
    y, bound = S.moe_few(x, ids, w, w13, w2, 0.0, 0.0)
    one = lambda e, v: w2[e] @ (S.silu(w13[e, :16] @ v) * (w13[e, 16:] @ v))
    np.testing.assert_allclose(y[0], 0.25 * one(0, x[0]) + 0.75 * one(3, x[0]))
    np.testing.assert_allclose(y[1], one(2, x[1]))
    assert not y[2].any() and not bound[2].any()
    assert (bound[:2] > 0).all()


def test_quantize_int8_rows():
    x = np.array([[127.0, -127.0, 0.5, 1.5], [0, 0, 0, 0], [1e-40, 0, 0, -1e-41], [2.54, 1.27, -0.01, 0.03]],
                 dtype=np.float32)
    q, s = S.quantize_int8(x)
    assert q[0].tolist() == [127, -127, 0, 2]      # halves to even
    assert q[1].tolist() == [0, 0, 0, 0] and s[1] == 1
    assert q[2].tolist() == [0, 0, 0, 0] and s[2] == 1
    assert q[3, 0] == 127 and abs(s[3] - 0.02) < 1e-8
