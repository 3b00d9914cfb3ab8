"""Router selection, the few-token expert layer and the 8-bit dense products
in 64-bit NumPy, from their definitions.

moe_gate         the k largest logits of a row (ties to the lowest index; -inf
                 and NaN masked) and their softmax, over the selected or all.
moe_gate_grad    the gradient of sum(dweights * weights) to the logits with the
                 selection held fixed.
moe_few          sum_j w_j W2_e (silu(G) * U), (G; U) = W13_e x, with a bound of
                 the float32 kernels' error from the sums' absolute values.
quantize_int8    rows in 8-bit integers, decided in float32 as the kernels do;
                 a row with a NaN or an infinity has the scale NaN.
"""
import numpy as np


def _masked(x):
    return ~(x > -np.inf)  # -inf and NaN


def moe_gate(logits, k, renormalize=True):
    """(weights float64 [T, k], ids int32 [T, k])."""
    x = np.asarray(logits, dtype=np.float64)
    key = np.where(_masked(x), -np.inf, x)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    v = np.take_along_axis(key, ids, axis=1)
    there = v > -np.inf
    m = np.where(there[:, :1], v[:, :1], 0.0)
    e = np.where(there, np.exp(np.where(there, v - m, 0.0)), 0.0)
    total = e.sum(1) if renormalize else np.exp(key - m).sum(1)
    w = e / np.where(total > 0, total, 1.0)[:, None]
    return w, np.where(there, ids, -1).astype(np.int32)


def fixed_weights(logits, ids, renormalize):
    """The weights as a function of the logits with the selection `ids` fixed."""
    x = np.asarray(logits, dtype=np.float64)
    there = ids >= 0
    v = np.where(there, np.take_along_axis(x, np.where(there, ids, 0), axis=1), -np.inf)
    key = np.where(_masked(x), -np.inf, x)
    m = np.where(there.any(1), key.max(1), 0.0)[:, None]
    e = np.exp(v - m)
    total = e.sum(1) if renormalize else np.exp(key - m).sum(1)
    return e / np.where(total > 0, total, 1.0)[:, None]


def moe_gate_grad(dweights, ids, logits, renormalize=True):
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    there = ids >= 0
    w = fixed_weights(x, ids, renormalize)
    g = np.where(there, dweights, 0.0)
    inner = (w * g).sum(1)
    if renormalize:
        p = np.zeros((T, E))
    else:
        key = np.where(_masked(x), -np.inf, x)
        m = np.where(there.any(1), key.max(1), 0.0)[:, None]
        p = np.exp(key - m)
        p = p / np.where(p.sum(1) > 0, p.sum(1), 1.0)[:, None]
    d = -p * inner[:, None]
    for t in range(T):
        for j in range(ids.shape[1]):
            if ids[t, j] >= 0:
                d[t, ids[t, j]] += w[t, j] * (g[t, j] - (inner[t] if renormalize else 0.0))
    return d


def silu(x):
    with np.errstate(over="ignore"):  # e^-x of a very negative x: the quotient is -0
        return x / (1.0 + np.exp(-x))


def moe_few(x, ids, weights, w13, w2, out_terms_eps, out_eps):
    """(y, bound): y float64 [T, H] and what a kernel with float32 sums may be
    off. w13 [E, 2F, H] and w2 [E, H, F] are dequantized float64 weights.
    out_terms_eps: relative error with which silu(G) * U is kept; out_eps: of
    the output type. A float32 sum of n products is off by (n + 8) 2^-24 times
    the sum of their absolute values at most."""
    x = np.asarray(x, dtype=np.float64)
    E, H, F = w2.shape
    gam = lambda n: (n + 8) * 2.0 ** -24
    y, err = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            p = w13[e] @ x[t]
            dp = gam(H) * (np.abs(w13[e]) @ np.abs(x[t])) + 2.0 ** -22 * np.abs(p)
            g, u, dg, du = p[:F], p[F:], dp[:F], dp[F:]
            h = silu(g) * u
            # |silu'| <= 1.1; exp, division and product round, exp's argument by up to |g| 2^-23
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + (8 + np.abs(g)) * 2.0 ** -23 * np.abs(h) \
                + out_terms_eps * np.abs(h)
            a = np.abs(w2[e])
            y[t] += weights[t, j] * (w2[e] @ h)
            err[t] += abs(weights[t, j]) * (a @ dh + (gam(F) + (ids.shape[1] + 4) * 2.0 ** -24) * (a @ (np.abs(h) + dh)))
    return y, err + out_eps * (np.abs(y) + err)


def quantize_int8(x):
    """(codes int8 [R, C], scales float32 [R]), every step in float32."""
    x = np.asarray(x, dtype=np.float32)
    s = (np.abs(x).max(1) * (np.float32(1) / np.float32(127))).astype(np.float32)
    s = np.where(s < np.float32(2.0 ** -126), np.float32(1), s).astype(np.float32)
    fine = np.isfinite(s)
    with np.errstate(invalid="ignore"):
        q = np.rint(x * (np.float32(1) / s).astype(np.float32)[:, None])
    q = np.where(fine[:, None], q, 0)  # unspecified
    return np.clip(q, -127, 127).astype(np.int8), np.where(fine, s, np.float32(np.nan)).astype(np.float32)


def gemm_int8(a, sa, b, sb, bias=None):
    y = (a.astype(np.float64) @ b.astype(np.float64).T) * sa.astype(np.float64)[:, None] * sb.astype(np.float64)
    return y if bias is None else y + bias.astype(np.float64)
