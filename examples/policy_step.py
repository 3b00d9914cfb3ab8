"""The last layer of a sampled policy and what its update needs.

    logits of the router = x Wr^T (8-bit product)   -> moe_gate_grouped: experts by sigmoid scores, balancing bias, groups
    routed = sum_j w_j W2_e SwiGLU(W13_e x)          -> moe_few_tokens_nvfp4
    shared = W2 SwiGLU(W13 x), 4-bit groups          -> linear_int4
    logits = (x + routed + shared) Wv^T, 4-bit groups -> linear_int4
    log p, entropy, alternatives of the sampled tokens -> token_logprobs, with the gradient to the logits, and the
    gradient of the experts' weights to the router's logits

Run: python examples/policy_step.py [tokens ...]
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_bit_quantize_amd as bsq  # noqa: E402


class Policy:
    def __init__(self, hidden=4096, ffn=1536, experts=64, topk=8, groups=8, group_k=4, vocabulary=32768, group=128, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        w = lambda *shape: torch.randn(*shape, generator=g, device=device) * 0.02
        self.topk, self.experts = topk, experts
        self.choose = dict(groups=groups, group_k=group_k)
        self.weigh = dict(score="sigmoid", renormalize=True, scale=2.5)
        per_expert = lambda rows, cols: [torch.cat(p) for p in
                                         zip(*(bsq.quantize_nvfp4(w(1, rows, cols).bfloat16(), "tensor")
                                               for _ in range(experts)))]
        self.w13, self.w2 = per_expert(2 * ffn, hidden), per_expert(hidden, ffn)
        self.wr = bsq.quantize_int8(w(experts, hidden))
        self.bias = torch.zeros(experts, device=device)
        self.s13 = bsq.quantize_int4(w(2 * ffn, hidden), group)
        self.s2 = bsq.quantize_int4(w(hidden, ffn), group)
        self.head = bsq.quantize_int4(w(vocabulary, hidden), group, symmetric=True)

    def gate(self, x):
        """(router logits, weights, expert ids) of the tokens."""
        logits = bsq.linear_int8(x, *self.wr, out_dtype=torch.float32)
        return (logits, *bsq.moe_gate_grouped(logits, self.topk, bias=self.bias, **self.choose, **self.weigh))

    def gate_gradient(self, logits, weights, ids, dweights):
        return bsq.moe_gate_grouped_backward(dweights, weights, ids, logits, **self.weigh)

    def balance(self, ids, rate=1e-3):
        """Experts with more than their share of the tokens become harder to choose."""
        load = torch.bincount(ids[ids >= 0].long(), minlength=self.experts).float()
        self.bias += rate * torch.sign(load.mean() - load)

    def shared(self, x):
        gate, up = bsq.linear_int4(x, *self.s13).float().chunk(2, 1)
        return bsq.linear_int4((torch.nn.functional.silu(gate) * up).to(x.dtype), *self.s2)

    def logits(self, x):
        """(logits [T, vocabulary], what the router did)."""
        router = self.gate(x)
        y = x + bsq.moe_few_tokens_nvfp4(x, router[2], router[1], *self.w13, *self.w2) + self.shared(x)
        return bsq.linear_int4(y, *self.head), router

    def step(self, x, targets, advantages, entropy_weight=0.01, top=5):
        """Loss -mean(advantage * log p + entropy_weight * H) of sampled tokens: (loss, dlogits, (log p, H, the
        alternatives' log p and ids), router)."""
        logits, router = self.logits(x)
        lp, entropy, stats, top_lp, top_ids = bsq.token_logprobs(logits, targets, top=top)
        loss = -(advantages * lp + entropy_weight * entropy).mean()
        n = x.shape[0]
        d = bsq.token_logprobs_backward(-advantages / n, torch.full_like(lp, -entropy_weight / n), logits, targets, stats,
                                        entropy)
        return loss, d, (lp, entropy, top_lp, top_ids), router


def main():
    tokens = [int(a) for a in sys.argv[1:]] or [1, 64]
    policy = Policy()
    for T in tokens:
        x = torch.randn(T, 4096, device="cuda").bfloat16()
        targets = torch.randint(0, 32768, (T,), device="cuda")
        advantages = torch.randn(T, device="cuda")
        for _ in range(3):
            out = policy.step(x, targets, advantages)
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            out = policy.step(x, targets, advantages)
        torch.cuda.synchronize()
        print(f"{T} tokens: loss {out[0].item():.4f}, {(time.perf_counter() - t) / 20 * 1e6:.0f} us a step")


if __name__ == "__main__":
    main()
