"""Products with 4-bit weights whose scales lie far apart, are zero, negative or tiny, on each way a product is laid
out: rows of x whole in LDS, slabs of K, tiles."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, log, t
from oracle import int4 as Q

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
OUT_EPS = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
ROWS = (2, 40, 100, 300)  # of x: few, slabs, tiles (float32; bf16), tiles


def dev(a, dtype=F32):
    x = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)
    return x, x.float().cpu().numpy().astype(np.float64)


def product(x, c, s, z, group, more=0.0):
    """Against the oracle's sums, its bound and half a step of float32; `more`: of what the bound has beside that."""
    log(f"linear_int4 scales {tuple(x.shape)} x {c.shape} group {group} {x.dtype}")
    xv = x.float().cpu().numpy().astype(np.float64)
    s = Q.bf16(s)
    y = bsq.linear_int4(x, t(c), torch.from_numpy(s).to(DEV).bfloat16(), None if z is None else t(z), out_dtype=F32)
    got = y.double().cpu().numpy()
    want, bound = Q.linear(xv, c, s, z)
    assert np.isfinite(got).all(), np.argwhere(~np.isfinite(got))[:4]
    off = np.abs(got - want)
    # values below the normal range of float32 are a step of 2^-149 apart
    tol = bound + OUT_EPS[F32] * (np.abs(want) + bound) + more + 2.0 ** -149
    assert (off <= tol).all(), (float((off / tol).max()), np.argwhere(off > tol)[:4])
    return got, want


def codes(rng, N, K, group, zeros=True):
    return (rng.integers(0, 256, (N, K // 2), dtype=np.uint8),
            rng.integers(0, 16, (N, K // group), dtype=np.uint8) if zeros else None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", ROWS)
def test_zero_scales_of_tiny_rows(M, group, dtype):
    """A row whose largest scale is below 2^-86, with groups of scale zero: 0 times their integers, no NaN."""
    rng = np.random.default_rng(M + group)
    N, K = 40, 1024
    c, z = codes(rng, N, K, group)
    s = np.exp2(rng.uniform(-9, -3, (N, K // group)))
    for n, top in enumerate((-60, -70, -86, -87, -95, -110, -126)):
        s[n] = np.exp2(top + rng.uniform(-1, 0, K // group))
        s[n, ::3] = 0.0
    s[7] = 0.0           # the whole row
    s[8, 1::2] = 0.0     # an ordinary row
    s[9, :-1] = 0.0
    s[10, 1:] = 0.0
    got, _ = product(dev(rng.standard_normal((M, K)), dtype)[0], c, s, z, group)
    assert (got[:, 7] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("M", ROWS)
def test_negative_scales(M, zeros, dtype):
    rng = np.random.default_rng(M)
    N, K, group = 50, 768, 64
    c, z = codes(rng, N, K, group, zeros)
    s = np.exp2(rng.uniform(-9, -3, (N, K // group))) * rng.choice([-1.0, 1.0], (N, K // group))
    product(dev(rng.standard_normal((M, K)), dtype)[0], c, s, z, group)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("group", [32, 128])
def test_large_activations_and_scales_far_apart(M, group):
    """bf16 x around 2^60, scales of 1 and 2^-64 and all between: sums and outputs are far from float32's end, whatever
    the order of the scales."""
    rng = np.random.default_rng(M + group)
    N, K = 48, 1024
    c, z = codes(rng, N, K, group)
    KG = K // group
    s = np.exp2(rng.uniform(-64, 0, (N, KG)))
    s[0] = np.where(np.arange(KG) % 2, 2.0 ** -64, 1.0)
    s[1] = np.where(np.arange(KG) % 2, 1.0, 2.0 ** -64)
    s[2] = np.exp2(-64.0 * np.arange(KG) / KG)
    s[3] = s[2, ::-1]
    s[4], s[4, 0] = 2.0 ** -64, 1.0
    s[5], s[5, 0] = 2.0 ** -120, 2.0 ** -40
    for size in (60, 100):
        product(dev(rng.standard_normal((M, K)) * 2.0 ** size, BF16)[0], c, s, z, group)


@pytest.mark.parametrize("dtype,far", [(BF16, 100), (F32, 80)])
@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("group", [32, 128])
def test_small_scales_beside_large_ones(M, group, dtype, far):
    """Where x is zero in the groups of a row's large scales, its outputs are those of the small ones, with all their
    bits: a scale of far less than 2^-64 of the row's largest is no other than itself."""
    rng = np.random.default_rng(M + group)
    N, K = 36, 1024
    c, z = codes(rng, N, K, group)
    KG = K // group
    s = np.exp2(rng.uniform(-far, -far + 8, (N, KG)))
    s[:, :KG // 2] = np.exp2(rng.uniform(-6, 0, (N, KG // 2)))
    s[1::2] = s[1::2, ::-1]
    x = rng.standard_normal((M, K))
    x[::2, :K // 2] = 0.0
    x[1::4, K // 2:] = 0.0
    got, want = product(dev(x, dtype)[0], c, s, z, group)
    small = (got[::2, ::2], want[::2, ::2])
    assert (np.abs(small[1]) < 2.0 ** (20 - far)).all() and (small[0] != 0).mean() > 0.99


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("K", [1024, 32768])
def test_largest_scales_of_float32_activations(M, K):
    """Scales just below 2^93 and small activations, all of one sign with the largest integers: the rows are brought to
    2^15 on the way, and 2^15 * 15 * 32768 * 2^93 is below 2^127."""
    rng = np.random.default_rng(M + K)
    N, group = 20, 128
    c, z = codes(rng, N, K, group)
    c[:4], z[:4] = 0xFF, 0
    s = np.exp2(rng.uniform(88, 92.9, (N, K // group)))
    x = rng.uniform(0.9, 1, (M, K)) * np.exp2(rng.integers(-100, 15, (M, 1)))
    product(dev(x)[0], c, s, z, group)
