"""The serving example with tokens that have fewer experts than slots: both ways
through the routed experts take the router's -1."""
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, log
from test_gpu_example import load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 300])
def test_slots_without_an_expert(T):
    log(f"expert layer with masked experts T={T}")
    layer = load().ExpertLayer(hidden=512, ffn=256, experts=8, topk=4, seed=1)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    x = torch.randn((T, 512), generator=g, device=DEV).bfloat16()
    logits = torch.randn((T, 8), generator=g, device=DEV)
    logits[0] = float("nan")             # no expert left
    logits[1, 2:] = -float("inf")        # two of four slots
    logits[T - 1, :7] = -float("inf")    # one
    w, ids = bsq.moe_gate(logits, 4)
    assert (ids < 0).sum(1)[[0, 1, T - 1]].tolist() == [4, 2, 3]
    full = layer.whole(ids)
    assert torch.equal(full[ids >= 0], ids[ids >= 0]) and full.min().item() >= 0 and full.max().item() < 8
    assert all(len(set(r)) == 4 for r in full.tolist())
    few = layer.routed_few(x, w, ids).float()
    many = layer.routed_many(x, w, ids).float()
    assert not few[0].any() and not many[0].any()
    # the grouped products quantize activations to 4 bits, row by row
    assert ((few - many).norm(dim=1)[1:] / many.norm(dim=1)[1:]).max().item() < 0.3


def test_a_row_of_nan_stays_in_its_row():
    T = 300                              # 1200 pairs: the grouped products
    layer = load().ExpertLayer(hidden=512, ffn=256, experts=8, topk=4, seed=1)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.randn((T, 512), generator=g, device=DEV).bfloat16()
    want = layer(x).float()
    x[7, 3] = float("nan")
    log("expert layer with a row of NaN")
    got = layer(x).float()
    assert got[7].isnan().all()
    keep = torch.arange(T, device=DEV) != 7
    assert ((got - want)[keep].norm() / want[keep].norm()).item() < 2.0 ** -8
