"""GPU parity of the router, the few-token expert layer and the 8-bit dense
products against their 64-bit oracle.

Tolerances are bounds, not measurements. Gate: a float32 softmax of k or E
terms whose exponents carry an error of 2^-24 of the distance to the maximum.
Expert layer: oracle.serving.moe_few's running bound. 8-bit products: the
integer sums are exact, so the output is off by its four float32 roundings and
the rounding of its type; codes match exactly."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log, t
from block_scaled_bit_quantize_amd._lib import MOE_FEW_MAX_PAIRS
from oracle import quant as Q
from oracle import serving as S

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
OUT_EPS = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def dev(a, dtype=F32):
    """float array -> device tensor of dtype, and the values it holds."""
    x = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)
    return x, x.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ router
def gate_case(rng, T, E, masked):
    x = rng.standard_normal((T, E)) * 2
    if masked:
        x[rng.random((T, E)) < masked] = -np.inf
    return x


def check_gate(x, k, renorm, dtype):
    xd, xv = dev(x, dtype)
    w, ids = bsq.moe_gate(xd, k, renormalize=renorm)
    wo, io = S.moe_gate(xv, k, renorm)
    np.testing.assert_array_equal(h(ids), io)
    finite = xv[np.isfinite(xv)]
    span = float(finite.max() - finite.min()) if finite.size else 0.0
    rel = (span + x.shape[1] + 16) * 2.0 ** -24
    np.testing.assert_allclose(h(w), wo, rtol=rel, atol=1e-37)
    g = np.random.default_rng(5).standard_normal(w.shape).astype(np.float32)
    d = bsq.moe_gate_backward(t(g), w, ids, xd, renormalize=renorm)
    assert d.dtype == dtype and d.shape == xd.shape
    do = S.moe_gate_grad(g.astype(np.float64), io, xv, renorm)
    size = np.abs(g).max(1, keepdims=True) if w.shape[1] else 0
    tol = 4 * (rel + k * 2.0 ** -24) * size + OUT_EPS[dtype] * np.abs(do)
    assert (np.abs(d.double().cpu().numpy() - do) <= tol).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (37, 64, 8), (130, 128, 8), (3, 256, 17), (17, 20, 3), (5, 1, 1),
                                   (9, 33, 33), (6, 63, 16), (4, 129, 64), (7, 257, 5), (3, 1000, 64), (2, 1024, 8)])
def test_gate(T, E, k, renorm, dtype):
    log(f"gate {T} {E} {k} {renorm} {dtype}")
    rng = np.random.default_rng(T * 1000 + E)
    check_gate(gate_case(rng, T, E, 0), k, renorm, dtype)
    check_gate(gate_case(rng, T, E, 0.6), k, renorm, dtype)


@pytest.mark.parametrize("E", [64, 100, 512])
def test_gate_special_rows(E):
    low = float(torch.finfo(F32).min)
    rows = np.zeros((9, E))
    rows[0] = -np.inf                      # nothing left
    rows[1] = -np.inf
    rows[1, E - 1] = 3.0                   # one left
    rows[2] = low                          # lowest finite value: not a mask
    rows[3] = np.where(np.arange(E) % 2, 0.0, -0.0)  # both zeros tie
    rows[4] = 7.0                          # all tie
    rows[5] = np.nan
    rows[6, 1::2] = np.nan                 # NaN masks its expert only
    rows[7] = low
    rows[7, 5] = 1.0                       # the others underflow
    rows[8] = np.linspace(-300, 300, E)
    log(f"gate special {E}")
    xd = t(rows.astype(np.float32))
    for renorm in (True, False):
        w, ids = bsq.moe_gate(xd, 4, renormalize=renorm)
        wo, io = S.moe_gate(rows.astype(np.float32), 4, renorm)
        np.testing.assert_array_equal(h(ids), io)
        np.testing.assert_allclose(h(w), wo, rtol=1e-4, atol=1e-37)  # exponents up to 600: 600 * 2^-23
        d = h(bsq.moe_gate_backward(torch.ones_like(w), w, ids, xd, renormalize=renorm))
        assert np.isfinite(d).all() and not d[0].any() and not d[5].any()


def test_gate_empty_and_aliases():
    w, ids = bsq.moe_gate(torch.empty((0, 64), device=DEV), 8)
    assert w.shape == (0, 8) and ids.shape == (0, 8)
    assert bsq.moe_gate_backward(w, w, ids, torch.empty((0, 64), device=DEV)).shape == (0, 64)
    # ids outside the range add nothing to the gradient
    x = torch.randn((3, 64), device=DEV)
    w, ids = bsq.moe_gate(x, 4)
    ids2 = ids.clone()
    ids2[1] = torch.tensor([-1, 64, 1 << 30, -(1 << 30)], dtype=torch.int32, device=DEV)
    d = bsq.moe_gate_backward(torch.ones_like(w) * torch.arange(4, device=DEV), w, ids2, x)
    assert not d[1].any() and d[0].any()


def test_gate_many_tokens_chain_into_route():
    T, E, k = 5003, 64, 8
    x = torch.randn((T, E), device=DEV)
    w, ids = bsq.moe_gate(x, k)
    io = S.moe_gate(x.cpu().numpy(), k)[1]
    np.testing.assert_array_equal(h(ids), io)
    _, seg, _ = bsq.route(ids, E)
    np.testing.assert_array_equal(h(seg), np.concatenate([[0], np.cumsum(np.bincount(io.ravel(), minlength=E))]))


def test_gate_gradient_against_differences():
    """The kernel's gradient against central differences of the 64-bit forward."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((4, 40)).astype(np.float32)
    k, eps = 6, 1e-5
    g = rng.standard_normal((4, k)).astype(np.float32)
    for renorm in (True, False):
        w, ids = bsq.moe_gate(t(x), k, renormalize=renorm)
        d = h(bsq.moe_gate_backward(t(g), w, ids, t(x), renormalize=renorm))
        i = h(ids)
        f = lambda z: (g * S.fixed_weights(z, i, renorm)).sum(1)
        for e in range(40):
            up, dn = x.astype(np.float64), x.astype(np.float64)
            up[:, e] += eps
            dn[:, e] -= eps
            # the difference's own error: third derivative eps^2, cancellation 2^-53 / eps
            np.testing.assert_allclose(d[:, e], (f(up) - f(dn)) / (2 * eps), atol=2e-5)


# ------------------------------------------------------------------ expert layer
def nvfp4_weights(rng, E, N, K):
    codes = rng.integers(0, 256, size=(E, N, K // 2), dtype=np.uint8)
    scales = rng.integers(0x20, 0x60, size=(E, N, K // 16), dtype=np.uint8)
    some = rng.random(scales.shape) < 0.02  # zero, subnormal and largest scales too
    scales[some] = rng.choice(np.array([0, 1, 7, 8, 0x7E], dtype=np.uint8), size=int(some.sum()))
    outer = (rng.random(E) * 2e-3 + 1e-3).astype(np.float32)
    return codes, scales, outer


def moe_case(T, H, F, E, k, dtype, seed, ids=None, scale=1.0):
    rng = np.random.default_rng(seed)
    w13, w2 = nvfp4_weights(rng, E, 2 * F, H), nvfp4_weights(rng, E, H, F)
    x, xv = dev(rng.standard_normal((T, H)) * scale, dtype)
    if ids is None:
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).reshape(T, k)
    ids = ids.astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    log(f"moe T={T} H={H} F={F} E={E} k={k} {dtype}")
    y = bsq.moe_few_tokens_nvfp4(x, t(ids), t(w), *map(t, w13), *map(t, w2))
    assert y.dtype == dtype and y.shape == x.shape
    deq = lambda a: Q.dequantize_nvfp4_f64(*a, Q.OUTER_TENSOR)
    ref, bound = S.moe_few(xv, ids, w.astype(np.float64), deq(w13), deq(w2), 2.0 ** -16 if dtype == BF16 else 2.0 ** -23,
                           OUT_EPS[dtype])
    off = np.abs(y.double().cpu().numpy() - ref)
    assert (off <= bound).all(), (off / np.maximum(bound, 1e-300)).max()
    return y, (x, t(ids), t(w), *map(t, w13), *map(t, w2))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,F,E,k", [(1, 256, 128, 8, 2), (1, 16, 16, 1, 1), (3, 272, 80, 5, 3), (7, 1040, 432, 20, 3),
                                       (16, 128, 48, 4, 2), (33, 144, 160, 40, 6), (64, 512, 96, 64, 8),
                                       (2, 48, 1040, 1024, 64)])
def test_moe_few(T, H, F, E, k, dtype):
    moe_case(T, H, F, E, min(k, E), dtype, seed=T + H)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [15, 16, 17, 63, 64, 65, 200])
def test_moe_few_one_expert_takes_all(n, dtype):
    ids = np.full((n, 2), 3)
    ids[:, 1] = np.arange(n) % 3
    moe_case(n, 80, 48, 6, 2, dtype, seed=n, ids=ids)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,k", [(1, 16), (1, 17), (2, 8), (5, 3), (16, 1), (17, 1)])
@pytest.mark.parametrize("H,F", [(16, 32), (4112, 48), (80, 256), (48, 272), (32, 1536), (64, 2048), (48, 2064),
                                 (32, 4096), (16, 4112)])
def test_moe_few_up_to_sixteen_pairs(T, k, H, F, dtype):
    """At and past 16 pairs, with inner lengths of one to eight spans of 256, of
    up to sixteen, and beyond; one id in five adds nothing."""
    rng = np.random.default_rng(T * k + F)
    E = 20 if H * F < 1 << 17 else 4
    ids = rng.integers(0, E, (T, k))
    ids[rng.random((T, k)) < 0.2] = -1
    moe_case(T, H, F, E, k, dtype, seed=H + F, ids=ids)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,F,E,k", [(2, 4112, 48, 3, 2), (9, 8208, 32, 4, 2), (1, 32, 8240, 4, 3), (20, 48, 4352, 3, 1),
                                       (40, 8448, 4128, 2, 1), (3, 16, 12304, 5, 2), (18, 16640, 16, 4, 1)])
def test_moe_few_rows_longer_than_the_registers(T, H, F, E, k, dtype):
    moe_case(T, H, F, E, k, dtype, seed=H + F)


def test_moe_few_small_repeats_bit_for_bit():
    _, args = moe_case(2, 528, 400, 16, 4, BF16, seed=8)
    y = bsq.moe_few_tokens_nvfp4(*args)
    for _ in range(3):
        assert torch.equal(y, bsq.moe_few_tokens_nvfp4(*args))


def test_moe_few_masked_pairs():
    ids = np.array([[-1, -1, -1], [2, -1, 7], [1 << 30, 0, 6], [6, 6, 6], [-5, 5, 64]])
    y, _ = moe_case(5, 96, 64, 8, 3, F32, seed=3, ids=ids)
    assert not y[0].any()
    y, _ = moe_case(4, 96, 64, 8, 2, BF16, seed=4, ids=np.full((4, 2), -1))
    assert not y.any()


def test_moe_few_pair_limit_and_empty():
    T = MOE_FEW_MAX_PAIRS // 8
    _, args = moe_case(T, 32, 16, 12, 8, BF16, seed=5)
    x, ids, w = args[:3]
    with pytest.raises(bsq.BsqError):
        bsq.moe_few_tokens_nvfp4(x.repeat(2, 1), ids.repeat(2, 1), w.repeat(2, 1), *args[3:])
    assert bsq.moe_few_tokens_nvfp4(x[:0], ids[:0], w[:0], *args[3:]).shape == (0, 32)


@pytest.mark.parametrize("scale", [1e-4, 300.0, 3e4])
def test_moe_few_magnitudes(scale):
    moe_case(4, 160, 96, 8, 2, BF16, seed=11, scale=scale)
    moe_case(4, 160, 96, 8, 2, F32, seed=12, scale=scale)


def test_moe_few_repeats_bit_for_bit_and_on_another_stream():
    _, args = moe_case(24, 512, 256, 16, 4, BF16, seed=6)
    y = bsq.moe_few_tokens_nvfp4(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        z = bsq.moe_few_tokens_nvfp4(*args)
    side.synchronize()
    assert torch.equal(y, z)


def test_moe_few_matches_the_chain():
    """The same experts through the many-token chain's products (which quantize
    the activations): as near as 4-bit activations allow."""
    T, H, F, E, k = 16, 512, 256, 8, 2
    rng = np.random.default_rng(9)
    mk = lambda *s: torch.from_numpy((rng.standard_normal(s) * 0.05).astype(np.float32)).to(DEV)
    w13, w2 = bsq.quantize_nvfp4(mk(E, 2 * F, H), "tensor"), bsq.quantize_nvfp4(mk(E, H, F), "tensor")
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(DEV).to(BF16)
    w, ids = bsq.moe_gate(mk(T, E) * 20, k)
    y = bsq.moe_few_tokens_nvfp4(x, ids, w, *w13, *w2).float()
    xq = bsq.quantize_nvfp4(x, "row", four_over_six=True)
    row, seg, pair = bsq.route(ids, E)
    h13 = bsq.grouped_gemm_nvfp4(*xq, *w13, seg, T * k, row_index=row)
    z = bsq.grouped_gemm_nvfp4(*bsq.swiglu_quantize_nvfp4(h13), *w2, seg, T * k, out_dtype=F32)
    want = (z[pair.long()].reshape(T, k, H) * w[:, :, None]).sum(1)
    assert ((y - want).norm() / want.norm()).item() < 0.25


# ------------------------------------------------------------------ 8-bit products
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,C", [(1, 16), (1, 4096), (3, 48), (2100, 272), (2048, 8192), (2050, 8208), (5, 32768),
                                 (70, 1536)])
def test_quantize_int8(R, C, dtype):
    log(f"quantize_int8 {R} {C} {dtype}")
    rng = np.random.default_rng(R + C)
    a = rng.standard_normal((R, C)) * np.exp(rng.uniform(-20, 20, (R, 1)))
    a[0] = 0
    if R > 2:
        a[2] = 1e-39  # scale below the normal range
    x, xv = dev(a, dtype)
    q, s = bsq.quantize_int8(x)
    qo, so = S.quantize_int8(xv)
    np.testing.assert_array_equal(h(s), so)
    np.testing.assert_array_equal(h(q), qo)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,F", [(1, 16), (3, 1536), (2100, 80), (4, 32768)])
def test_swiglu_quantize_int8(R, F, dtype):
    log(f"swiglu_quantize_int8 {R} {F} {dtype}")
    rng = np.random.default_rng(R + F)
    x, xv = dev(rng.standard_normal((R, 2 * F)) * 3, dtype)
    q, s = bsq.swiglu_quantize_int8(x)
    v = S.silu(xv[:, :F]) * xv[:, F:]
    so = np.abs(v).max(1) / 127
    np.testing.assert_allclose(h(s), so, rtol=(16 + 8) * 2.0 ** -23)  # exp's argument up to 16
    # a code may be the other neighbour only where the value lies within that error of the middle
    assert (np.abs(h(q).astype(np.float64) - v / so[:, None]) <= 0.5 + 127 * 32 * 2.0 ** -23).all()


def int8_case(M, N, K, out_dtype, bias, seed, extreme=False):
    rng = np.random.default_rng(seed)
    a = rng.integers(-128, 128, size=(M, K), dtype=np.int8)
    b = rng.integers(-128, 128, size=(N, K), dtype=np.int8)
    if extreme:
        a[:], b[:] = -128, -128
    sa = np.exp(rng.uniform(-5, 5, M)).astype(np.float32)
    sb = np.exp(rng.uniform(-5, 5, N)).astype(np.float32)
    bi = (rng.standard_normal(N) * 100).astype(np.float32) if bias else None
    log(f"gemm_int8 {M} {N} {K} {out_dtype} bias={bias}")
    y = bsq.gemm_int8(t(a), t(sa), t(b), t(sb), bias=None if bi is None else t(bi), out_dtype=out_dtype)
    ref = S.gemm_int8(a, sa, b, sb, bi)
    prod = S.gemm_int8(a, sa, b, sb)
    tol = 4 * 2.0 ** -24 * np.abs(prod) + (2.0 ** -24 + OUT_EPS[out_dtype]) * np.abs(ref)
    off = np.abs(y.double().cpu().numpy() - ref)
    assert (off <= tol).all(), float((off / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 4096, 4096), (1, 33, 48), (7, 100, 1040), (16, 64, 64), (17, 65, 80),
                                   (33, 17, 512), (50, 250, 7168), (64, 128, 128), (65, 127, 144), (128, 128, 128),
                                   (129, 1, 16), (200, 300, 272), (256, 256, 1024), (257, 513, 640), (1000, 259, 1536),
                                   (700, 2048, 256)])
def test_gemm_int8(M, N, K, out_dtype):
    int8_case(M, N, K, out_dtype, bias=(M + N) % 2 == 0, seed=M + N + K)


@pytest.mark.parametrize("M", [3, 130])
def test_gemm_int8_largest_sums(M):
    """Every product 128 * 128 at the largest K: the sum stays inside 32 bits."""
    int8_case(M, 40, 131056, F32, False, seed=1, extreme=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 100, 4096), (4, 48, 32768), (5, 4096, 1040), (60, 96, 7168), (300, 260, 528)])
def test_linear_int8_is_the_two_calls(M, N, K, dtype):
    rng = np.random.default_rng(M)
    x, _ = dev(rng.standard_normal((M, K)), dtype)
    b = t(rng.integers(-127, 128, size=(N, K), dtype=np.int8))
    sb = t(rng.random(N).astype(np.float32))
    bias = t(rng.random(N).astype(np.float32))
    log(f"linear_int8 {M} {N} {K} {dtype}")
    for od in (BF16, F32):
        y = bsq.linear_int8(x, b, sb, bias=bias, out_dtype=od)
        assert torch.equal(y, bsq.gemm_int8(*bsq.quantize_int8(x), b, sb, bias=bias, out_dtype=od))
    assert bsq.linear_int8(x, b, sb).dtype == dtype


def test_int8_empty():
    b = torch.zeros((8, 32), dtype=torch.int8, device=DEV)
    sb = torch.ones(8, device=DEV)
    assert bsq.linear_int8(torch.empty((0, 32), device=DEV), b, sb).shape == (0, 8)
    assert bsq.linear_int8(torch.ones((3, 32), device=DEV), b[:0], sb[:0]).shape == (3, 0)
    q, s = bsq.quantize_int8(torch.empty((0, 32), device=DEV))
    assert q.shape == (0, 32) and s.shape == (0,)


# ------------------------------------------------------------------ refusals
def test_bindings_refuse():
    f = lambda *s: torch.zeros(s, device=DEV)
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    bad = [
        lambda: bsq.moe_gate(f(4, 8).half(), 2),
        lambda: bsq.moe_gate(f(4, 8), 9),                       # k > E
        lambda: bsq.moe_gate(f(4, 8), 0),
        lambda: bsq.moe_gate(f(8, 4).t(), 2),                   # not contiguous
        lambda: bsq.moe_gate(f(4, 8).cpu(), 2),
        lambda: bsq.moe_gate(f(2, 1025), 2),
        lambda: bsq.moe_gate(f(8), 2),
        lambda: bsq.moe_gate_backward(f(4, 2), f(4, 2), i32(4, 3), f(4, 8)),
        lambda: bsq.moe_gate_backward(f(4, 2), f(4, 2), i32(4, 2).long(), f(4, 8)),
        lambda: bsq.quantize_int8(f(4, 24)),
        lambda: bsq.quantize_int8(f(4, 32784)),
        lambda: bsq.quantize_int8(f(4, 32).double()),
        lambda: bsq.swiglu_quantize_int8(f(4, 33)),
        lambda: bsq.swiglu_quantize_int8(f(4, 48)),
        lambda: bsq.gemm_int8(i8(4, 32), f(4), i8(8, 48), f(8)),
        lambda: bsq.gemm_int8(i8(4, 24), f(4), i8(8, 24), f(8)),
        lambda: bsq.gemm_int8(i8(4, 32), f(3), i8(8, 32), f(8)),
        lambda: bsq.gemm_int8(i8(4, 32), f(4), i8(8, 32), f(8), bias=f(4)),
        lambda: bsq.gemm_int8(i8(4, 32), f(4), i8(8, 32), f(8), out_dtype=torch.float16),
        lambda: bsq.linear_int8(f(4, 32), i8(8, 32).to(torch.uint8), f(8)),
        lambda: bsq.linear_int8(f(4, 32).t(), i8(8, 32), f(8)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(bsq.BsqError):
            call()
            pytest.fail(f"call {n} was accepted")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    good = dict(x=f(2, 32), topk_ids=i32(2, 2), topk_weights=f(2, 2), w13_codes=u8(4, 32, 16), w13_scales=u8(4, 32, 2),
                w13_outer=f(4), w2_codes=u8(4, 32, 8), w2_scales=u8(4, 32, 1), w2_outer=f(4))
    bsq.moe_few_tokens_nvfp4(**good)
    for name, v in [("x", f(2, 48)), ("x", f(2, 32).half()), ("topk_ids", i32(2, 2).long()), ("topk_ids", i32(1, 2)),
                    ("topk_weights", f(2, 3)), ("w13_codes", u8(4, 30, 16)), ("w13_scales", u8(4, 32, 1)),
                    ("w13_outer", f(3)), ("w2_codes", u8(3, 32, 8)), ("w2_scales", i8(4, 32, 1)),
                    ("w2_outer", f(4).double())]:
        with pytest.raises(bsq.BsqError):
            bsq.moe_few_tokens_nvfp4(**{**good, name: v})
            pytest.fail(f"{name} was accepted")


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(66, 70, 528), (300, 65, 2064), (130, 1030, 384), (2050, 1026, 208), (4100, 4099, 80),
                                   (4096, 4096, 128), (8200, 515, 96)])
def test_gemm_int8_tiles(M, N, K, out_dtype):
    """Every tile size, with rows of outputs that are not whole 16-byte pieces."""
    int8_case(M, N, K, out_dtype, bias=N % 2 == 1, seed=K)


@pytest.mark.parametrize("T,H,F,E,k", [(3, 4096, 1536, 16, 4), (2, 7168, 64, 4, 2), (2, 8208, 48, 4, 2), (5, 6160, 2064, 4, 2),
                                       (1, 64, 8208, 3, 1), (128, 64, 64, 8, 8)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_moe_few_long_rows(T, H, F, E, k, dtype):
    """Rows at and past what the streams keep in registers."""
    moe_case(T, H, F, E, k, dtype, seed=H + F)


def test_moe_few_skewed_experts():
    """Some experts take several passes, most one, some none."""
    rng = np.random.default_rng(4)
    ids = np.stack([rng.choice(40, size=6, replace=False, p=(lambda p: p / p.sum())(np.arange(1, 41) ** -1.5))
                    for _ in range(150)])
    moe_case(150, 96, 80, 40, 6, BF16, seed=4, ids=ids)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1540, 2570, 48), (1001, 4099, 144), (385, 12160, 272), (4600, 900, 1040)])
def test_gemm_int8_a_few_more_tiles_than_cus(M, N, K, out_dtype):
    int8_case(M, N, K, out_dtype, bias=K > 200, seed=M + K)
