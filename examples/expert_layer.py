"""An expert layer for serving: router, NVFP4 experts and a shared expert in
8-bit integers.

    logits = x Wr^T (8-bit product)        -> moe_gate: top-k experts and weights
    routed = sum_j w_j W2_e SwiGLU(W13_e x) -> moe_few_tokens_nvfp4 for a few tokens,
                                              the grouped NVFP4 products for many
    shared = W2 SwiGLU(W13 x)               -> linear_int8, swiglu_quantize_int8, gemm_int8

Run: python examples/expert_layer.py [tokens ...]
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_bit_quantize_amd as bsq  # noqa: E402


class ExpertLayer:
    def __init__(self, hidden=4096, ffn=1536, experts=64, topk=8, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        w = lambda *shape: torch.randn(*shape, generator=g, device=device) * 0.02
        self.hidden, self.ffn, self.experts, self.topk = hidden, ffn, experts, topk
        # routed experts: NVFP4, one outer scale each (drawn and quantized one by one)
        per_expert = lambda rows, cols: [torch.cat(p) for p in
                                         zip(*(bsq.quantize_nvfp4(w(1, rows, cols).bfloat16(), "tensor")
                                               for _ in range(experts)))]
        self.w13 = per_expert(2 * ffn, hidden)
        self.w2 = per_expert(hidden, ffn)
        # router and shared expert: 8-bit integers, a scale for each output channel
        self.wr = bsq.quantize_int8(w(experts, hidden))
        self.s13 = bsq.quantize_int8(w(2 * ffn, hidden))
        self.s2 = bsq.quantize_int8(w(hidden, ffn))

    def gate(self, x):
        """(logits, weights, expert ids) of the tokens."""
        logits = bsq.linear_int8(x, *self.wr, out_dtype=torch.float32)
        return (logits, *bsq.moe_gate(logits, self.topk))

    def gate_gradient(self, logits, weights, ids, dweights):
        """Gradient of the experts' weights to the router's logits."""
        return bsq.moe_gate_backward(dweights, weights, ids, logits)

    def shared(self, x):
        h13 = bsq.linear_int8(x, *self.s13)
        return bsq.gemm_int8(*bsq.swiglu_quantize_int8(h13), *self.s2, out_dtype=x.dtype)

    def routed_few(self, x, weights, ids):
        return bsq.moe_few_tokens_nvfp4(x, ids, weights, *self.w13, *self.w2)

    def whole(self, ids):
        """ids for route, which takes distinct experts alone: a slot without one (-1: logits that are masked or NaN)
        gets one that its token has not chosen, whose row is left out of the sum."""
        none = ids < 0
        chosen = torch.zeros((ids.shape[0], self.experts + 1), dtype=torch.int8, device=ids.device)
        chosen.scatter_(1, torch.where(none, self.experts, ids).long(), 1)
        left = torch.argsort(chosen[:, :self.experts], dim=1, stable=True)  # those not chosen first
        return torch.where(none, left.gather(1, (none.cumsum(1) - 1).clamp(min=0)).int(), ids)

    def routed_many(self, x, weights, ids):
        T, k = ids.shape
        rows, seg, pair = bsq.route(self.whole(ids), self.experts)
        xq = bsq.quantize_nvfp4(x, "row", four_over_six=True)
        h13 = bsq.grouped_gemm_nvfp4(*xq, *self.w13, seg, T * k, row_index=rows)
        z = bsq.grouped_gemm_nvfp4(*bsq.swiglu_quantize_nvfp4(h13), *self.w2, seg, T * k, out_dtype=torch.float32)
        z = z[pair.long()].reshape(T, k, -1) * weights[:, :, None]
        return z.masked_fill((ids < 0)[:, :, None], 0.0).sum(1).to(x.dtype)

    def __call__(self, x):
        _, weights, ids = self.gate(x)
        # the streamed experts; above, tiles of 256 rows fill up. Top 8 of 64 experts, streamed and grouped: 156 and
        # 457 us for 256 pairs, 207 and 489 for 1024, 350 and 526 for 2048, which is as many as are streamed
        few = ids.numel() <= 1024
        return (self.routed_few if few else self.routed_many)(x, weights, ids) + self.shared(x)


def main(tokens):
    layer = ExpertLayer()
    for T in tokens:
        x = torch.randn(T, layer.hidden, device="cuda").bfloat16()
        y = layer(x)
        logits, w, ids = layer.gate(x)
        few = layer.routed_few(x, w, ids).float() if ids.numel() <= 2048 else None
        many = layer.routed_many(x, w, ids).float()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(20):
            layer(x)
        torch.cuda.synchronize()
        us = (time.perf_counter() - t) / 20 * 1e6
        line = f"{T} tokens: {us:.0f} us a layer, finite {bool(torch.isfinite(y).all())}"
        if few is not None:
            line += f", streamed against grouped products (4-bit activations): {((few - many).norm() / many.norm()).item():.3f}"
        print(line, flush=True)
    d = layer.gate_gradient(logits, w, ids, torch.ones_like(w))
    print(f"gradient to the router's logits: {tuple(d.shape)}, row sums at most {d.sum(1).abs().max().item():.1e}")


if __name__ == "__main__":
    main([int(a) for a in sys.argv[1:]] or [1, 8, 64, 1024])
