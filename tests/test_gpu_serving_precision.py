"""How exactly the expert layer keeps small values beside large ones.

The weights pick single values: gate rows the largest, x_0 = 8, up row i the
value x_i, and W2 is the identity, so y_i = silu(8) x_i. x falls from 2^-1 to
2^-36 of x_0. Documented: bfloat16 x is exact down to 2^-31 of the largest,
float32 x and h = silu(G) U have 22 bits down to 2^-16 of it, and what is
smaller is off by 2^-39 of the largest at most."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log, t
from oracle import serving as S

pytestmark = pytest.mark.gpu

ONE, SCALE_ONE = 2, 0x38  # 1.0 in E2M1 and in E4M3


def picking(rows, cols, at):
    """NVFP4 [1, rows, cols] with a single 1.0 in each row, at column at[row]."""
    codes = np.zeros((1, rows, cols // 2), dtype=np.uint8)
    for r, c in enumerate(at):
        codes[0, r, c // 2] = ONE << (4 * (c % 2))
    return codes, np.full((1, rows, cols // 16), SCALE_ONE, dtype=np.uint8), np.ones(1, dtype=np.float32)


@pytest.mark.parametrize("tokens", [1, 20])  # W2 with its sum in one launch, and apart
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_small_beside_large(dtype, tokens):
    log(f"expert layer, small beside large {tokens} {dtype}")
    n = 256                                # one span: one scale for the whole row
    rng = np.random.default_rng(0)
    x = 8.0 * 2.0 ** (-1 - 35 * np.arange(n) / (n - 1)) * (1 + rng.random(n)) / 2
    x[0] = 8.0
    xd = torch.from_numpy(x.astype(np.float32)).to(DEV).to(dtype)
    xv = xd.double().cpu().numpy()
    w13 = picking(2 * n, n, [0] * n + list(range(n)))
    w2 = picking(n, n, range(n))
    y = bsq.moe_few_tokens_nvfp4(xd.repeat(tokens, 1), t(np.zeros((tokens, 1), np.int32)), t(np.ones((tokens, 1), np.float32)),
                                 *map(t, w13), *map(t, w2))
    act = S.silu(np.float64(8.0))
    ref = act * xv
    largest_h = act * 8.0
    of_x = np.where(xv >= 8 * 2.0 ** -16, 2.0 ** -22 * xv, 2.0 ** -39 * 8)
    if dtype == torch.bfloat16:
        of_x = np.where(xv >= 8 * 2.0 ** -31, 0, 2.0 ** -39 * 8)
    of_h = np.where(ref >= largest_h * 2.0 ** -16, 2.0 ** -22 * ref, 2.0 ** -39 * largest_h)
    # exponential, division and products of the SwiGLU, and the rounded sums of the two terms
    rounding = (16 + 8) * 2.0 ** -23 * ref
    tol = (act * of_x + of_h + rounding) * (1 + 2.0 ** -8) + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * ref
    off = np.abs(y.double().cpu().numpy() - ref[None])
    assert (off <= tol).all(), (off / tol).max()
