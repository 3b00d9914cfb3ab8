"""The grouped router, the 4-bit products and the token log probabilities as they are used together, against plain
float64 arithmetic on the same weights."""
import os
import sys

import numpy as np
import pytest
import torch

from _gpu_util import DEV, h, log
from oracle import int4 as Q
from oracle import logprob as L
from oracle import router as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def values(q):
    return torch.from_numpy(Q.values(h(q[0]), q[1].float().cpu().numpy(), None if q[2] is None else h(q[2])))


@pytest.fixture(scope="module")
def policy():
    from policy_step import Policy
    return Policy(hidden=512, ffn=256, experts=32, topk=4, groups=4, group_k=2, vocabulary=1003, group=64)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_step(policy, T):
    log(f"policy step {T}")
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, 512, generator=g).to(DEV)
    targets = torch.randint(0, 1003, (T,), generator=g).to(DEV)
    if T > 1:
        targets[1] = -100
    adv = torch.randn(T, generator=g).to(DEV)
    logits, (rl, w, ids) = policy.logits(x)
    loss, d, (lp, entropy, top_lp, top_ids), router = policy.step(x, targets, adv)
    # the router, from its own logits
    wo, io = R.group_gate(h(rl), 4, h(policy.bias), 4, 2, 2, "sigmoid", True, 2.5)
    np.testing.assert_array_equal(h(ids), io)
    np.testing.assert_allclose(h(w), wo, rtol=2.0 ** -17)
    # the shared expert and the head: float32 sums (bounds of the oracle), through SwiGLU
    x64 = x.double().cpu()
    h13, b13 = Q.linear(x64.numpy(), h(policy.s13[0]), policy.s13[1].float().cpu().numpy(), h(policy.s13[2]))
    gate, up = np.split(h13, 2, axis=1)
    bg, bu = np.split(b13, 2, axis=1)
    act = gate / (1 + np.exp(-gate)) * up
    # |silu'| <= 1.1; silu and the product are off by a few roundings
    off = 1.1 * bg * np.abs(up) + np.abs(gate) * bu + 2.0 ** -21 * np.abs(act) + bg * bu
    w2 = values(policy.s2).numpy()
    want, bound = Q.linear(act, h(policy.s2[0]), policy.s2[1].float().cpu().numpy(), h(policy.s2[2]))
    got = policy.shared(x).double().cpu().numpy()
    assert (np.abs(got - want) <= bound * 1.01 + off @ np.abs(w2).T + 2.0 ** -24 * np.abs(want)).all()
    # log probabilities and the gradient, from the logits
    t = h(targets)
    wl, we, wt, wi = L.token_logprobs(h(logits), t, 5)
    np.testing.assert_array_equal(h(top_ids), wi)
    for a, b in ((lp, wl), (entropy, we), (top_lp, wt)):
        np.testing.assert_allclose(h(a), b, rtol=2.0 ** -17, atol=2.0 ** -17)
    n = T
    do = L.gradient(-h(adv).astype(np.float64) / n, np.full(T, -0.01 / n), h(logits), t)
    np.testing.assert_allclose(h(d), do, rtol=0, atol=2.0 ** -17 * (np.abs(h(adv)).max() + 1) / n)
    np.testing.assert_allclose(loss.item(), -(h(adv) * wl + 0.01 * we).mean(), rtol=1e-5, atol=1e-5)
    # the loss moves with the logits as the gradient says: a step of s along it changes it by s |d|^2, to second order
    # (curvature of the loss below 4 max|adv| |d|^2 s^2), in float32 sums of about 10
    step = 0.25
    import block_scaled_bit_quantize_amd as bsq
    moved = bsq.token_logprobs((logits + step * d).contiguous(), targets)
    loss2 = -(adv * moved[0] + 0.01 * moved[1]).mean().item()
    size = float((d.double() ** 2).sum())
    assert abs((loss2 - loss.item()) - step * size) <= 4 * (float(adv.abs().max()) + 1) * step ** 2 * size + 1e-4
    dw = torch.randn(w.shape, generator=g).to(DEV)
    dg = policy.gate_gradient(rl, w, ids, dw)
    want = R.group_gate_grad(h(dw), io, h(rl), "sigmoid", True, 2.5)
    np.testing.assert_allclose(h(dg), want, rtol=0, atol=2.0 ** -16 * 2.5 * float(dw.abs().max()))


def test_balance_and_routing(policy):
    """The ids feed route, and the bias moves against the load."""
    import block_scaled_bit_quantize_amd as bsq
    x = torch.randn(64, 512, device=DEV)
    before = policy.bias.clone()
    _, _, ids = policy.gate(x)
    rows, seg, _ = bsq.route(ids, 32)
    load = (seg[1:] - seg[:-1]).float()
    policy.balance(ids)
    torch.testing.assert_close(policy.bias - before, 1e-3 * torch.sign(load.mean() - load))
    policy.bias.copy_(before)
