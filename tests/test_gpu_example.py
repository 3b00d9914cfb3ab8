"""The serving example's expert layer, small: its parts against the 64-bit oracle
and its two ways through the routed experts against each other."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log
from oracle import quant as Q
from oracle import serving as S

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T", [1, 9, 300])
def test_expert_layer(T):
    log(f"expert layer T={T}")
    layer = load().ExpertLayer(hidden=512, ffn=256, experts=8, topk=4, seed=1)
    x = torch.randn((T, 512), device=DEV).bfloat16()
    xv = x.double().cpu().numpy()
    # logits: one product of 8-bit codes
    q, s = S.quantize_int8(xv)
    logits, w, ids = layer.gate(x)
    np.testing.assert_allclose(h(logits), S.gemm_int8(q, s, h(layer.wr[0]), h(layer.wr[1])), rtol=2 ** -21, atol=1e-12)
    wo, io = S.moe_gate(h(logits), 4)
    np.testing.assert_array_equal(h(ids), io)
    # routed experts
    y = layer.routed_few(x, w, ids)
    deq = lambda p: Q.dequantize_nvfp4_f64(*map(h, p), Q.OUTER_TENSOR)
    ref, bound = S.moe_few(xv, io, h(w).astype(np.float64), deq(layer.w13), deq(layer.w2), 2.0 ** -16, 2.0 ** -8)
    assert (np.abs(y.double().cpu().numpy() - ref) <= bound).all()
    many = layer.routed_many(x, w, ids).double()
    assert ((y.double() - many).norm() / many.norm()).item() < 0.25  # the grouped products quantize activations to 4 bits
    # the layer is the sum of its parts, whichever way it takes
    few = ids.numel() <= 1024
    assert torch.equal(layer(x), (y if few else layer.routed_many(x, w, ids)) + layer.shared(x))
    # the router's gradient sums to zero over the experts of a token: the weights sum to one
    d = layer.gate_gradient(logits, w, ids, torch.randn_like(w))
    assert d.sum(1).abs().max().item() < 1e-5 and torch.count_nonzero(d, dim=1).max().item() <= 4
