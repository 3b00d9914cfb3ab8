"""The router's special rows in bfloat16, whose selection is a path of its own
(key and index in one word)."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log
from oracle import serving as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [8, 64, 100, 128, 256, 512])
def test_gate_special_rows(E):
    low = float(torch.finfo(torch.bfloat16).min)
    rows = np.zeros((10, E))
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
    rows[9] = np.where(np.arange(E) % 3, -2.0 ** -130, 2.0 ** -133)  # subnormal, of both signs
    log(f"gate special bf16 {E}")
    xd = torch.from_numpy(rows.astype(np.float32)).to(DEV).bfloat16()
    xv = xd.float().cpu().numpy()
    for renorm in (True, False):
        w, ids = bsq.moe_gate(xd, 4, renormalize=renorm)
        wo, io = S.moe_gate(xv, 4, renorm)
        np.testing.assert_array_equal(h(ids), io)
        np.testing.assert_allclose(h(w), wo, rtol=1e-4, atol=1e-37)  # exponents up to 600: 600 * 2^-23
        g = np.ones((10, 4)) * np.array([1.0, -2.0, 3.0, 0.5])
        gd = torch.from_numpy(g.astype(np.float32)).to(DEV)
        d = bsq.moe_gate_backward(gd, w, ids, xd, renormalize=renorm).float().cpu().numpy()
        do = S.moe_gate_grad(g, io, xv, renorm)
        assert np.isfinite(d).all() and not d[0].any() and not d[5].any()
        assert (np.abs(d - do) <= 2.0 ** -8 * np.abs(do) + 3 * 4e-4).all()
