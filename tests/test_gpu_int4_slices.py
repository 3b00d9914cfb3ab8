"""Products with 4-bit weights in several slices of weights and of rows, by each of the tiles whole and in parts of K,
and what float32 activations keep of their bits."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, log, t
from oracle import int4 as Q

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def around(borders, end):
    """The places next to each border, the first and the last ones."""
    at = {i for b in (0, *borders, end) for i in range(b - 3, b + 3)}
    return np.array(sorted(i for i in at if 0 <= i < end))


def check_sampled(M, N, K, group, dtype, rows=(), columns=(), bias=True):
    log(f"linear_int4 {M} x {N} x {K} group {group} {dtype}")
    rng = np.random.default_rng(M + N + K)
    c = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = Q.bf16(np.exp2(rng.uniform(-9, -3, (N, K // group))))
    z = rng.integers(0, 16, (N, K // group), dtype=np.uint8)
    x = torch.from_numpy(rng.standard_normal((M, K), dtype=np.float32)).to(DEV).to(dtype)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    y = bsq.linear_int4(x, t(c), torch.from_numpy(s).to(DEV).bfloat16(), t(z), None if b is None else t(b), out_dtype=F32)
    assert torch.isfinite(y).all()
    m, n = around(rows, M), np.unique(np.concatenate((around(columns, N), rng.integers(0, N, 8))))
    m = np.unique(np.concatenate((m, rng.integers(0, M, 8))))
    want, bound = Q.linear(x[torch.from_numpy(m).to(DEV)].double().cpu().numpy(), c[n], s[n], z[n], None if b is None else b[n])
    got = y.cpu().numpy().astype(np.float64)[np.ix_(m, n)]
    off, tol = np.abs(got - want), bound + 2.0 ** -24 * (np.abs(want) + bound)
    assert (off <= tol).all(), (float((off / tol).max()), np.argwhere(off > tol)[:4])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [200, 1300])
def test_slices_of_weights(M, dtype):
    """128 MiB of unpacked weights at a time: 4096 rows of 16384, the last slice of 108."""
    check_sampled(M, 8300, 16384, 64, dtype, (128, 192, 256, 1024), (4096, 8192))


@pytest.mark.parametrize("group", [32, 128])
def test_slices_of_rows_and_of_weights(group):
    """64 MiB of float32 activations in two parts at a time: 512 rows of 32768, then 88; 2048 rows of weights, then 52."""
    check_sampled(600, 2100, 32768, group, F32, (128, 192, 256, 384, 512), (2048,))


def test_slices_of_rows():
    check_sampled(4500, 300, 4096, 64, F32, (4096,), (128, 256))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K,group", [(130, 140, 384, 64), (1500, 4200, 512, 64), (2049, 4352, 512, 32),
                                         (5000, 4200, 256, 128), (3001, 8195, 128, 128), (1536, 4096, 4096, 128)])
def test_whole_tiles(M, N, K, group, dtype):
    """Sizes whose least time is that of one of the tiles without a split of K: in bf16 128 x 128, 256 x 128 and
    256 x 256, in float32 128 x 128, 192 x 128 and 128 x 256."""
    check_sampled(M, N, K, group, dtype, (128, 192, 256, 384, M // 256 * 256, M // 192 * 192),
                  (128, 256, N // 256 * 256), bias=K < 512)


# ------------------------------------------------------------------ what float32 activations keep
@pytest.mark.parametrize("M", [2, 40, 100])
def test_small_values_beside_a_large_one(M):
    """A row's largest value meets a weight of zero: its other values are off by 2^-22 of themselves, or by 2^-39 of the
    largest (2^-40 for a half step, at 2^15 for a value just below twice its power of two)."""
    rng = np.random.default_rng(M)
    N, K, group = 40, 512, 64
    c = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    z = rng.integers(0, 16, (N, K // group), dtype=np.uint8)
    s = Q.bf16(np.exp2(rng.uniform(-4, 0, (N, K // group))))
    c[:, 100] = (c[:, 100] & 0xF0) | z[:, 200 // group]  # value 200 of every row of weights is 0
    for up in (10, 20, 30, 45):
        log(f"linear_int4 float32 {M} rows, one value 2^{up}")
        x = rng.standard_normal((M, K)).astype(np.float32)
        x[:, 200] = 2.0 ** up * rng.uniform(1, 2, M)
        y = bsq.linear_int4(t(x), t(c), torch.from_numpy(s).to(DEV).bfloat16(), t(z)).double().cpu().numpy()
        rest = x.astype(np.float64)
        top = np.abs(rest).max(1, keepdims=True)
        rest[:, 200] = 0.0
        want, _ = Q.linear(rest, c, s, z)
        q, zz, ss = Q.parts(c, s, z)
        size = ((q + zz) * np.abs(ss)).reshape(N, -1)
        # sums in float32, of terms among which the large one is (its group's sums of q x and of z x cancel)
        _, bound = Q.linear(x, c, s, z)
        lost = 2.0 ** -39 * top * size.sum(1)
        assert (np.abs(y - want) <= bound + lost).all()
        if M > 64:  # tiles sum (q - z) x: nothing of the large value enters
            w = Q.values(c, s, z)
            _, small = Q.linear(rest, c, s, z)
            lost = 2.0 ** -39 * top * np.abs(w).sum(1)
            assert (np.abs(y - want) <= small + lost).all()


@pytest.mark.parametrize("M", [2, 40, 100])
def test_rows_of_tiny_values(M):
    """Rows whose largest value is below 2^-112: values are off by 2^-22 of themselves or by 2^-151 (2^-149 is the least
    float32 there is), whichever is more."""
    rng = np.random.default_rng(M)
    N, K, group = 40, 512, 64
    c = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    z = rng.integers(0, 16, (N, K // group), dtype=np.uint8)
    s = Q.bf16(np.exp2(rng.uniform(60, 64, (N, K // group))))
    x = (rng.standard_normal((M, K)) * np.exp2(rng.integers(-146, -108, (M, 1)))).astype(np.float32)
    x[0] = 0.0
    log(f"linear_int4 float32 {M} rows of tiny values")
    y = bsq.linear_int4(t(x), t(c), torch.from_numpy(s).to(DEV).bfloat16(), t(z)).double().cpu().numpy()
    want, bound = Q.linear(x, c, s, z)
    lost = 2.0 ** -151 * np.abs(Q.values(c, s, z)).sum(1)
    assert (np.abs(y - want) <= bound + 2.0 ** -24 * (np.abs(want) + bound) + lost).all()
    assert (y[0] == 0).all()
