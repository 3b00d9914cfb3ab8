"""The 8-bit products at the limits of their dispatch, and gates where the
SwiGLU's exponential overflows."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log
from oracle import serving as S

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# Rows are quantized inside the product up to 16 rows and 16384 (bfloat16) or 8192 (float32) values: the limits
# themselves, single rows that fill them, inner lengths with fewer steps than waves, and the first sizes past them.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(16, 70, 1024), (1, 33, 16384), (16, 50, 512), (1, 40, 8192), (15, 17, 16), (3, 20, 112),
                                   (16, 1, 16), (17, 40, 512), (16, 33, 1040), (16, 33, 528), (1, 33, 16400), (1, 40, 8208)])
def test_linear_int8_is_the_two_calls_at_its_limits(M, N, K, dtype):
    log(f"linear_int8 {M} {N} {K} {dtype}")
    rng = np.random.default_rng(M + K)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(DEV).to(dtype)
    if M > 2:
        x[M - 1] *= 1e3
        x[M // 2] = 0
    b = torch.from_numpy(rng.integers(-127, 128, size=(N, K), dtype=np.int8)).to(DEV)
    sb = torch.from_numpy(rng.random(N).astype(np.float32)).to(DEV)
    q, s = S.quantize_int8(x.float().cpu().numpy())
    for od in (BF16, F32):
        y = bsq.linear_int8(x, b, sb, out_dtype=od)
        assert torch.equal(y, bsq.gemm_int8(*bsq.quantize_int8(x), b, sb, out_dtype=od))
        ref = S.gemm_int8(q, s, h(b), h(sb))
        eps = 2.0 ** -8 if od == BF16 else 2.0 ** -24
        assert (np.abs(y.double().cpu().numpy() - ref) <= (4 * 2.0 ** -24 + eps) * np.abs(ref)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R", [3, 2100])  # a workgroup a row, a wave a row
def test_swiglu_quantize_int8_gates_of_any_size(R, dtype):
    """silu goes to 0 from below where e^-g overflows, and to g above."""
    log(f"swiglu_quantize_int8 large gates {R} {dtype}")
    F = 272
    rng = np.random.default_rng(R)
    gate = rng.choice(np.array([-3e38, -1e4, -200, -104, -90, -88, -80, -20, 0, 20, 88, 1e3, 1e4]), (R, F))
    up = rng.standard_normal((R, F))
    gate[0] = -200.0                      # nothing but zeros
    x = torch.from_numpy(np.concatenate([gate, up], 1).astype(np.float32)).to(DEV).to(dtype)
    xv = x.double().cpu().numpy()
    q, s = bsq.swiglu_quantize_int8(x)
    g, u = xv[:, :F], xv[:, F:]
    with np.errstate(over="ignore"):
        v = S.silu(g) * u
    # the exponential's argument is off by |g| 2^-23 of it and the few operations by units of 2^-23; what is below the
    # normal range may go to 0
    dv = (np.minimum(np.abs(g), 200) + 8) * 2.0 ** -23 * np.abs(v) + 2.0 ** -126 * (1 + np.abs(u))
    so = np.abs(v).max(1) / 127
    one = so < 2.0 ** -126                # scale 1, codes 0
    assert one[0] and not one[1:].any()
    sv = h(s).astype(np.float64)
    assert sv[0] == 1 and not h(q)[0].any()
    assert (np.abs(sv - so)[1:] <= (dv.max(1) / 127 + 2.0 ** -22 * so)[1:]).all()
    assert (np.abs(h(q) * sv[:, None] - v)[1:] <= (0.5 * sv[:, None] * (1 + 127 * 2.0 ** -22) + dv)[1:]).all()
