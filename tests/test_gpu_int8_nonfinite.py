"""NaN and infinities in the rows of the 8-bit products: such a row's scale and
outputs are NaN, whichever kernel quantizes it, and the rows beside it keep
their bits."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log
from oracle import serving as S

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def rows_with(R, C, dtype, seed):
    """(rows, the same with NaN and infinities in some, those rows)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((R, C), generator=g, device=DEV).to(dtype)
    y = x.clone()
    put = [(0, C - 1, NAN), (R // 2, 0, INF), (R - 1, C // 2, -INF)]
    if R > 6:
        put += [(1, c, NAN) for c in range(C)] + [(3, 0, INF), (3, 1, NAN), (4, 5, -NAN)]
    for r, c, v in put:
        y[r, c] = v
    bad = torch.zeros(R, dtype=torch.bool)
    bad[[r for r, _, _ in put]] = True
    return x, y, bad.to(DEV)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,C", [(1, 16), (3, 4096), (7, 1040), (2500, 272), (2050, 8208)])
def test_quantize_int8(R, C, dtype):
    log(f"quantize_int8 with NaN {R} {C} {dtype}")
    x, y, bad = rows_with(R, C, dtype, R)
    q0, s0 = bsq.quantize_int8(x)
    q, s = bsq.quantize_int8(y)
    assert s[bad].isnan().all()
    assert torch.equal(s[~bad], s0[~bad]) and torch.equal(q[~bad], q0[~bad])
    np.testing.assert_array_equal(h(s), S.quantize_int8(y.float().cpu().numpy())[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,F", [(1, 16), (9, 1536), (2500, 80)])
def test_swiglu_quantize_int8(R, F, dtype):
    log(f"swiglu_quantize_int8 with NaN {R} {F} {dtype}")
    g = torch.Generator(device=DEV)
    g.manual_seed(R)
    x = torch.randn((R, 2 * F), generator=g, device=DEV).to(dtype)
    q0, s0 = bsq.swiglu_quantize_int8(x)
    y = x.clone()
    put = [(0, 3, NAN)] if R == 1 else [(0, 3, NAN), (2, F + 5, NAN), (3, 1, -INF), (R - 1, 7, INF)]
    for r, c, v in put:
        y[r, c] = v
    if R > 5:
        y[5, 0] = y[5, F] = 3e38  # the product overflows
        put.append((5, 0, INF))
    bad = torch.zeros(R, dtype=torch.bool, device=DEV)
    bad[[r for r, _, _ in put]] = True
    q, s = bsq.swiglu_quantize_int8(y)
    assert s[bad].isnan().all()
    assert torch.equal(s[~bad], s0[~bad]) and torch.equal(q[~bad], q0[~bad])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 33, 4096), (3, 48, 1040), (9, 70, 528), (20, 65, 1040), (60, 33, 272), (300, 130, 528)])
def test_linear_int8(M, N, K, dtype):
    log(f"linear_int8 with NaN {M} {N} {K} {dtype}")
    x, y, bad = rows_with(M, K, dtype, M)
    b = torch.randint(-127, 128, (N, K), device=DEV, dtype=torch.int8)
    sb, bias = torch.rand(N, device=DEV), torch.rand(N, device=DEV)
    for od in (BF16, F32):
        want, got = bsq.linear_int8(x, b, sb, bias, out_dtype=od), bsq.linear_int8(y, b, sb, bias, out_dtype=od)
        assert got[bad].isnan().all()
        assert torch.equal(got[~bad], want[~bad])
        two = bsq.gemm_int8(*bsq.quantize_int8(y), b, sb, bias=bias, out_dtype=od)
        assert two[bad].isnan().all() and torch.equal(two[~bad], got[~bad])
