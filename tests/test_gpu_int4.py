"""4-bit groups and their products against the 64-bit oracle: codes, scales and zero
points exactly, products within the oracle's bound and half a step of the output's type."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log, t
from oracle import int4 as Q

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
OUT_EPS = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def dev(a, dtype=F32):
    x = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)
    return x, x.float().cpu().numpy().astype(np.float64)


def weights(rng, N, K, group, zeros):
    """Random codes, bf16 scales of both signs of exponent, zero points: host arrays and device tensors."""
    c = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = Q.bf16(np.exp2(rng.uniform(-9, -3, (N, K // group))))
    z = rng.integers(0, 16, (N, K // group), dtype=np.uint8) if zeros else None
    return (c, s, z), (t(c), torch.from_numpy(s).to(DEV).bfloat16(), t(z) if zeros else None)


# ------------------------------------------------------------------ quantizer
def check_quant(w, group, symmetric, dtype):
    log(f"quantize_int4 {w.shape} {group} {symmetric} {dtype}")
    wd, wv = dev(w, dtype)
    codes, scales, zeros = bsq.quantize_int4(wd, group, symmetric)
    assert codes.dtype == torch.uint8 and scales.dtype == BF16 and (zeros is None) == symmetric
    c, s, z = Q.quantize(wv, group, symmetric)
    np.testing.assert_array_equal(scales.float().cpu().numpy(), s)
    fine = np.isfinite(s)
    got = h(codes).reshape(*s.shape, -1)
    np.testing.assert_array_equal(got[fine], c.reshape(*s.shape, -1)[fine])
    if not symmetric:
        np.testing.assert_array_equal(h(zeros)[fine], z[fine])
        assert (h(zeros) <= 15).all()
    for out in (F32, BF16):
        v = bsq.dequantize_int4(codes, scales, zeros, out_dtype=out)
        want = torch.from_numpy(Q.values(h(codes), s, None if zeros is None else h(zeros)).astype(np.float32)).to(out)
        assert torch.equal(v.cpu().nan_to_num(7.0), want.nan_to_num(7.0)) and v.dtype == out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (3, 64, 64), (5, 128, 128), (7, 96, 32), (129, 320, 64), (37, 1152, 128),
                                       (1, 32768, 128), (513, 224, 32)])
def test_quantize(N, K, group, symmetric, dtype):
    rng = np.random.default_rng(N + K)
    check_quant(rng.standard_normal((N, K)) * 0.02, group, symmetric, dtype)
    check_quant(np.abs(rng.standard_normal((N, K))), group, symmetric, dtype)
    check_quant(-np.abs(rng.standard_normal((N, K))) * 1e30, group, symmetric, dtype)
    w = np.where(rng.random((N, K)) < 0.05, rng.standard_normal((N, K)) * 20, rng.standard_normal((N, K)))
    check_quant(w * np.exp2(rng.integers(-120, 100, (N, 1))), group, symmetric, dtype)


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_ties(symmetric):
    """Values at and one unit next to the middle between two codes, at scales that are and are not powers of two."""
    rows = []
    for s in (1.0, 1.0078125, 0.3828125, 3.0, 1.9921875):
        mid = (np.arange(-7, 7) + 0.5) * s
        lows, highs = np.nextafter(mid.astype(np.float32), -np.inf), np.nextafter(mid.astype(np.float32), np.inf)
        for m in (mid, lows, highs):
            row = np.zeros(64)
            row[0], row[1] = (7 * s, -7 * s) if symmetric else (8 * s, -7 * s)
            row[2:16] = m
            row[32], row[33] = (-7 * s, 0) if symmetric else (15 * s, 0)
            row[34:48] = m
            rows.append(row)
    check_quant(np.array(rows), 32, symmetric, F32)
    check_quant(np.array(rows), 64, symmetric, F32)


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_special(symmetric):
    w = np.zeros((8, 128))
    w[1, 5] = np.nan
    w[2, 5] = np.inf
    w[3, 100] = -np.inf
    w[4, :] = 1e-40
    w[5, :] = 2e-38
    w[6, :] = 3e38
    w[6, ::2] = -3e38
    w[7, 64:] = -1e-3
    check_quant(w, 32, symmetric, F32)
    check_quant(w, 128, symmetric, BF16)


def test_quantize_large():
    """Past 2^31 values: the last rows against the same rows quantized by themselves."""
    N, K = (1 << 16) + 3, 32768
    w = torch.empty((N, K), dtype=BF16, device=DEV)
    w[:] = torch.randn((1, K), device=DEV).to(BF16)
    w[-5:] = torch.randn((5, K), device=DEV).to(BF16)
    log("quantize_int4 large")
    codes, scales, zeros = bsq.quantize_int4(w, 32)
    for rows in (slice(0, 2), slice(N - 5, N)):
        for a, b in zip((codes, scales, zeros), bsq.quantize_int4(w[rows].contiguous(), 32)):
            assert torch.equal(a[rows], b)
    v = bsq.dequantize_int4(codes, scales, zeros, out_dtype=BF16)
    assert torch.equal(v[-5:], bsq.dequantize_int4(codes[-5:], scales[-5:], zeros[-5:], out_dtype=BF16))


# ------------------------------------------------------------------ products
def check_linear(rng, M, N, K, group, zeros, dtype, out=None, bias=False, outliers=True):
    log(f"linear_int4 {M} x {N} x {K} group {group} zeros {zeros} {dtype} -> {out} bias {bias}")
    (c, s, z), w = weights(rng, N, K, group, zeros)
    x = rng.standard_normal((M, K))
    if outliers:
        x = np.where(rng.random(x.shape) < 1e-2, x * 20, x)
    xd, xv = dev(x, dtype)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    y = bsq.linear_int4(xd, *w, bias=t(b) if bias else None, out_dtype=out)
    assert y.dtype == (out or dtype) and y.shape == (M, N)
    want, bound = Q.linear(xv, c, s, z, b)
    off = np.abs(y.double().cpu().numpy() - want)
    tol = bound + OUT_EPS[y.dtype] * (np.abs(want) + bound)
    assert (off <= tol).all(), (float((off / tol).max()), np.argwhere(off > tol)[:4])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 1, 128), (2, 17, 256), (5, 100, 1152), (16, 33, 640), (3, 515, 4096),
                                   (1, 4096, 512), (13, 48, 2048)])
def test_few(M, N, K, group, dtype):
    rng = np.random.default_rng(M * 100 + N + K)
    check_linear(rng, M, N, K, group, True, dtype)
    check_linear(rng, M, N, K, group, False, dtype, bias=True)


@pytest.mark.parametrize("M,N,K,group", [(1, 5, 32, 32), (4, 20, 96, 32), (16, 31, 992, 32), (2, 9, 64, 64), (7, 65, 192, 64),
                                         (3, 18, 4160, 64), (1, 40, 32768, 128), (2, 24, 32736, 32), (9, 16, 16384, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_ragged(M, N, K, group, dtype):
    """K that no chunk of 128 divides, rows of x that fill LDS, several launches."""
    rng = np.random.default_rng(M + N + K)
    check_linear(rng, M, N, K, group, True, dtype, bias=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("M,N,K", [(17, 16, 128), (31, 100, 2048), (48, 515, 4096), (64, 33, 8192), (192, 70, 1152),
                                   (16, 50, 8192), (130, 4100, 512)])
def test_slabs(M, N, K, group, dtype):
    """More rows than share a workgroup's LDS whole: slabs of K, one or several, one launch or several."""
    rng = np.random.default_rng(M + N + K)
    check_linear(rng, M, N, K, group, True, dtype)
    check_linear(rng, M, N, K, group, False, dtype, BF16, bias=True)


def test_slabs_of_many_channels():
    """More channels than the slabs' sums are kept for at a time: the columns around the border and the last ones."""
    rng = np.random.default_rng(11)
    M, N, K, group = 64, 66000, 8192, 128
    (c, s, z), w = weights(rng, N, K, group, True)
    x, xv = dev(rng.standard_normal((M, K)), BF16)
    log(f"linear_int4 {M} x {N} x {K}")
    y = bsq.linear_int4(x, *w, out_dtype=F32)
    for n in (slice(0, 20), slice(65500, 65560), slice(N - 20, N)):
        want, bound = Q.linear(xv, c[n], s[n], z[n])
        assert (np.abs(y[:, n].double().cpu().numpy() - want) <= bound + 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F32, BF16)])
def test_other_output_type(dtype, out):
    rng = np.random.default_rng(1)
    check_linear(rng, 3, 70, 384, 64, True, dtype, out)
    check_linear(rng, 200, 70, 384, 64, True, dtype, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(49, 64, 128), (64, 130, 1152), (65, 257, 512), (100, 1000, 2176), (129, 512, 4096),
                                   (300, 4099, 256), (1001, 515, 640)])
def test_many(M, N, K, group, dtype):
    rng = np.random.default_rng(M + N + K)
    check_linear(rng, M, N, K, group, True, dtype)
    check_linear(rng, M, N, K, group, False, dtype, bias=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K,group", [(50, 33, 32, 32), (70, 40, 96, 32), (130, 200, 992, 32), (64, 64, 64, 64), (90, 77, 192, 64),
                                         (257, 129, 4128, 32), (80, 1030, 32768, 128)])
def test_many_ragged(M, N, K, group, dtype):
    rng = np.random.default_rng(M + N + K)
    check_linear(rng, M, N, K, group, True, dtype, bias=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_tiles(dtype):
    """Enough rows for the largest tiles, several slices of rows (float32) and of weights."""
    rng = np.random.default_rng(7)
    check_linear(rng, 4100, 2050, 256, 128, True, dtype, bias=True)
    check_linear(rng, 2050, 4100, 192, 32, True, dtype)
    check_linear(rng, 700, 2200, 16384, 64, False, dtype)


def test_rows_do_not_mix():
    """A row of x gives the same bits alone and in a batch of few; NaN and infinite rows keep to themselves."""
    rng = np.random.default_rng(3)
    _, w = weights(rng, 200, 1024, 128, True)
    x, _ = dev(rng.standard_normal((8, 1024)), BF16)
    y = bsq.linear_int4(x, *w)
    for m in range(8):
        assert torch.equal(bsq.linear_int4(x[m:m + 1], *w)[0], y[m])
    for M in (8, 200):
        x, _ = dev(rng.standard_normal((M, 1024)), BF16)
        y = bsq.linear_int4(x, *w)
        bad = x.clone()
        bad[3, 77], bad[5, 1000], bad[6, 0] = float("nan"), float("inf"), -float("inf")
        z = bsq.linear_int4(bad, *w)
        keep = [m for m in range(M) if m not in (3, 5, 6)]
        assert torch.equal(z[keep], y[keep])
        assert not torch.isfinite(z[[3, 5, 6]]).any()


def test_nan_scale_is_one_output():
    rng = np.random.default_rng(4)
    _, (c, s, z) = weights(rng, 40, 512, 128, True)
    s[7, 2] = float("nan")
    for M in (2, 100):
        y = bsq.linear_int4(torch.randn((M, 512), device=DEV), c, s, z)
        assert torch.isnan(y[:, 7]).all()
        assert torch.isfinite(y[:, [n for n in range(40) if n != 7]]).all()


def test_quantized_weights_end_to_end():
    rng = np.random.default_rng(5)
    w = torch.from_numpy(rng.standard_normal((300, 768)).astype(np.float32) * 0.02).to(DEV)
    x = torch.from_numpy(rng.standard_normal((4, 768)).astype(np.float32)).to(DEV)
    for symmetric in (True, False):
        q = bsq.quantize_int4(w, 64, symmetric)
        v = bsq.dequantize_int4(*q).double().cpu()
        y = bsq.linear_int4(x, *q).double().cpu()
        _, bound = Q.linear(x.cpu().numpy(), h(q[0]), q[1].float().cpu().numpy(), None if symmetric else h(q[2]))
        want = x.double().cpu() @ v.t()
        assert ((y - want).abs().numpy() <= bound + 2.0 ** -24 * np.abs(want.numpy())).all()


def test_empty_and_refusals():
    c = torch.zeros((8, 64), dtype=torch.uint8, device=DEV)
    s = torch.ones((8, 1), dtype=BF16, device=DEV)
    z = torch.zeros((8, 1), dtype=torch.uint8, device=DEV)
    x = torch.zeros((3, 128), dtype=BF16, device=DEV)
    assert bsq.linear_int4(x[:0], c, s, z).shape == (0, 8)
    assert bsq.linear_int4(x, c[:0], s[:0], z[:0]).shape == (3, 0)
    assert bsq.dequantize_int4(c[:0], s[:0]).shape == (0, 128)
    q = bsq.quantize_int4(x[:0])
    assert q[0].shape == (0, 64) and q[1].shape == (0, 1)
    for bad in ((x.half(), c, s, z), (x[:, :64], c, s, z), (x[0], c, s, z), (x, c.int(), s, z), (x, c, s.float(), z),
                (x, c, s, z.int()), (x, c, s, z[:4]), (x, c, s[:4], z), (x, c[:, :40], s, z), (x.cpu(), c, s, z),
                (x, c, s, z, torch.zeros(7, device=DEV)), (x, c, s, z, torch.zeros(8, device=DEV, dtype=BF16)),
                (x, c, s, z, None, torch.float16)):
        with pytest.raises(bsq.BsqError):
            bsq.linear_int4(*bad)
    for bad in (dict(group=16), dict(group=96), dict(group=256)):
        with pytest.raises(bsq.BsqError):
            bsq.quantize_int4(torch.zeros((4, 192), device=DEV), **bad)
    with pytest.raises(bsq.BsqError):
        bsq.quantize_int4(torch.zeros((4, 128), device=DEV).half())
    with pytest.raises(bsq.BsqError):
        bsq.dequantize_int4(c, s, z, out_dtype=torch.float16)


@pytest.mark.parametrize("M,dtype", [(1, BF16), (3, F32), (40, BF16), (60, F32), (500, BF16)])
def test_stream_and_graph(M, dtype):
    rng = np.random.default_rng(M)
    _, w = weights(rng, 300, 1024, 64, True)
    x = torch.randn((M, 1024), device=DEV).to(dtype)
    step = lambda: bsq.linear_int4(x, *w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y = step()
    torch.cuda.current_stream().wait_stream(s)
    for i in range(4):
        x.copy_(torch.randn((M, 1024), device=DEV))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_neighbours_are_left_alone():
    """Nothing is written around the output: a larger buffer keeps its other bytes."""
    from block_scaled_bit_quantize_amd import _lib
    lib = _lib.load_library()
    rng = np.random.default_rng(6)
    for M, N in ((3, 21), (100, 77)):
        _, (c, s, z) = weights(rng, N, 256, 64, True)
        x = torch.randn((M, 256), device=DEV).to(BF16)
        buf = torch.full((M * N + 128,), 5.0, dtype=BF16, device=DEV)
        wsb = lib.bsq_linear_int4_workspace(M, N, 256, 64, 1)
        ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=DEV)
        assert lib.bsq_linear_int4(x.data_ptr(), 1, c.data_ptr(), s.data_ptr(), z.data_ptr(), 64, None, M, N, 256,
                                   buf[61:].data_ptr(), 1, ws.data_ptr(), wsb, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(buf[61:61 + M * N].view(M, N), bsq.linear_int4(x, c, s, z))
        assert (buf[:61] == 5).all() and (buf[61 + M * N:] == 5).all()
