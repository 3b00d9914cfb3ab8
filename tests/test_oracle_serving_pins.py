"""Further pins of the 64-bit oracle of the serving operators (no GPU)."""
import numpy as np

from oracle import serving as S


def test_gemm_int8_against_python_integers():
    rng = np.random.default_rng(3)
    a = rng.integers(-128, 128, (5, 48), dtype=np.int8)
    b = rng.integers(-128, 128, (7, 48), dtype=np.int8)
    a[0], b[0] = -128, -128
    sa, sb = 2.0 ** rng.integers(-3, 4, 5).astype(np.float32), 2.0 ** rng.integers(-3, 4, 7).astype(np.float32)
    bias = rng.integers(-9, 9, 7).astype(np.float32)
    y = S.gemm_int8(a, sa, b, sb, bias)
    for m in range(5):
        for n in range(7):
            want = sum(int(p) * int(q) for p, q in zip(a[m], b[n])) * float(sa[m]) * float(sb[n]) + float(bias[n])
            assert y[m, n] == want  # powers of two: every step is exact


def test_quantize_int8_on_a_grid():
    rng = np.random.default_rng(4)
    q = rng.integers(-127, 128, (20, 32)).astype(np.int8)
    q[:, 0] = 127
    step = 2.0 ** rng.integers(-20, 20, 20)
    codes, s = S.quantize_int8(q * step[:, None])
    np.testing.assert_array_equal(codes, q)
    np.testing.assert_allclose(s, step, rtol=2.0 ** -23)


def test_moe_few_bound_holds_float32_and_not_a_planted_rounding():
    rng = np.random.default_rng(5)
    H, F = 256, 64
    x = rng.standard_normal((4, H)).astype(np.float32)
    w13, w2 = rng.standard_normal((2, 2 * F, H)), rng.standard_normal((2, H, F))
    w13, w2 = w13.astype(np.float32), w2.astype(np.float32)
    ids = np.array([[0, 1], [1, 0], [1, -1], [0, 1]], dtype=np.int32)
    w = rng.random((4, 2)).astype(np.float32)
    y, bound = S.moe_few(x, ids, w.astype(np.float64), w13.astype(np.float64), w2.astype(np.float64), 2.0 ** -23, 2.0 ** -24)

    def layer(cut):
        out = np.zeros((4, H), dtype=np.float32)
        for t in range(4):
            for j in range(2):
                e = ids[t, j]
                if e < 0:
                    continue
                g, u = w13[e, :F] @ x[t], w13[e, F:] @ x[t]
                out[t] += w[t, j] * (w2[e] @ cut((g / (np.float32(1) + np.exp(-g)) * u).astype(np.float32)))
        return out

    def to_bf16(v):
        b = v.view(np.uint32)
        return ((b + 0x7FFF + (b >> 16 & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)

    assert (np.abs(layer(lambda v: v) - y) <= bound).all()
    assert (np.abs(layer(to_bf16) - y) > bound).any()
