"""Weights in 4-bit groups and products with them, in 64-bit NumPy from the
definitions.

quantize    codes 0..15, bf16 scales and zero points of groups along K.
values      what they stand for, (q - z) * s.
linear      x W^T + bias with a bound on the error of float32 sums.
"""
import numpy as np


def bf16(x):
    """float32 values of float64/float32 input, rounded to float32 and then to bf16, half to even."""
    with np.errstate(over="ignore"):
        f = np.asarray(x).astype(np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(f), np.float32(np.nan), r)


def quantize(w, group, symmetric):
    """w [N, K] -> (codes u8 [N, K/2], scales float32 [N, K/group] of bf16 values, zeros u8 or None)."""
    N, K = w.shape
    g = np.asarray(w, dtype=np.float64).reshape(N, K // group, group)
    lo, hi = np.minimum(g.min(2), 0), np.maximum(g.max(2), 0)  # NaN where one is
    s = bf16(np.maximum(-lo, hi) / 7 if symmetric else (hi - lo) / 15)
    s = np.where(np.isfinite(g).all(2), s, np.float32(np.nan))
    s = np.where(s < 2.0 ** -126, np.float32(1), s)
    s64 = s.astype(np.float64)
    with np.errstate(invalid="ignore"):
        z = np.full(s.shape, 8.0) if symmetric else np.clip(np.rint(-lo / s64), 0, 15)
        q = np.clip(np.rint(g / s64[:, :, None]) + z[:, :, None], 0, 15)
        z, q = np.nan_to_num(z).astype(np.uint8), np.nan_to_num(q).astype(np.uint8).reshape(N, K // 2, 2)
    return (q[:, :, 0] | q[:, :, 1] << 4).astype(np.uint8), s, None if symmetric else z


def parts(codes, scales, zeros):
    """(q, z, s) float64, q [N, groups, group], z and s [N, groups, 1]."""
    N, KG = scales.shape
    q = np.stack((codes & 15, codes >> 4), -1).reshape(N, KG, -1).astype(np.float64)
    z = np.full((N, KG), 8.0) if zeros is None else zeros.astype(np.float64)
    return q, z[:, :, None], scales.astype(np.float64)[:, :, None]


def values(codes, scales, zeros=None):
    q, z, s = parts(codes, scales, zeros)
    return ((q - z) * s).reshape(codes.shape[0], -1)


def linear(x, codes, scales, zeros=None, bias=None):
    """(y, bound) float64 [M, N]. bound: what float32 sums may be off by. A group's sums of q x and of z x (or of
    (q - z) x) are exact products added one after the other, two parts of each for float32 activations, then a sum
    over groups and parts of K: one rounding, or one cut at the same place, for each addition, 2^-23 of at most the sum
    of the terms' sizes. (Two additions a value of a group; the third covers the cut of float32 activations to 22 bits,
    2^-22 of the sum of the terms' sizes.)"""
    x = np.asarray(x, dtype=np.float64)
    q, z, s = parts(codes, scales, zeros)
    N, KG, group = q.shape
    w = ((q - z) * s).reshape(N, -1)
    size = ((q + z) * np.abs(s)).reshape(N, -1)
    y = x @ w.T
    bound = (3 * group + KG + 32) * 2.0 ** -23 * (np.abs(x) @ size.T)
    if bias is not None:
        y = y + bias
        bound = bound + 2.0 ** -23 * np.abs(bias)
    return y, bound
