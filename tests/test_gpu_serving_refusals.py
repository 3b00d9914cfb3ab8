"""Refusals of the router's binding before it allocates anything."""
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [-1, 0, 9, 65, 1 << 50])
def test_gate_k(k):
    log(f"gate refuses k={k}")
    for E in (8, 128):
        if 1 <= k <= min(E, 64):
            continue
        with pytest.raises(bsq.BsqError):
            bsq.moe_gate(torch.zeros((4, E), device=DEV), k)
    with pytest.raises(bsq.BsqError):
        bsq.moe_gate(torch.zeros((0, 8), device=DEV), k)
