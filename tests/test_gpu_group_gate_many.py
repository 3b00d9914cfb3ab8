"""The grouped router at many tokens, at numbers of experts that do not fill its lanes or take a wave a row."""
import numpy as np
import pytest
import torch

from test_gpu_group_gate import check

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("E,k,groups,group_k", [(144, 6, 1, 1), (160, 6, 8, 3), (192, 8, 6, 2), (240, 12, 1, 1), (257, 4, 1, 1),
                                                (320, 8, 8, 4), (384, 8, 1, 1), (384, 6, 12, 4), (512, 8, 8, 4),
                                                (512, 10, 1, 1), (768, 16, 64, 20), (1024, 8, 16, 4)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_tokens_of_many_experts(E, k, groups, group_k, dtype):
    rng = np.random.default_rng(E + groups)
    T = 2049
    x = rng.standard_normal((T, E)) * 2
    x[::7] = np.round(x[::7])  # many ties
    x[5::11, :E // 2] = -np.inf
    bias = rng.standard_normal(E) * 0.05
    check(x, k, dtype, bias, groups, group_k, 2, "sigmoid", True, 2.5)
    check(x, k, dtype, None, groups, group_k, 1, "softmax", False)
