"""What the router, the few-token expert layer and the 8-bit dense products cost.

Four kinds of pass:
  gate    top-k expert selection over router logits; with "grad" also the gradient to the logits
  moe     a whole NVFP4 expert layer for a few tokens: gate and up projection, SwiGLU, down projection, weighted sum
  linear  a dense layer in 8-bit integers: rows quantized with a scale each, product with per-channel scales
  mlp     the same as a gated MLP (the shared expert beside the routed ones): two products around a SwiGLU

The sizes are those of the benchmark's workloads (16384 or 65536 tokens, hidden 4096 or 7168, 64 or 128 experts of
1536 or 2048, top-8) and ragged ones around them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token in a decode step: latency only
        {"name": "gate_1", "kind": "gate", "T": 1, "E": 64, "k": 8, "dtype": "f32", "renorm": True, "masked": 0,
         "grad": False},
        # the router of the 16384-token training step, forward and backward
        {"name": "gate_16384", "kind": "gate", "T": 16384, "E": 64, "k": 8, "dtype": "f32", "renorm": True,
         "masked": 0, "grad": True},
        # the 65536-token step's router, bf16 logits, probabilities over all experts, some experts masked (-inf)
        {"name": "gate_65536_bf16", "kind": "gate", "T": 65536, "E": 128, "k": 8, "dtype": "bf16", "renorm": False,
         "masked": 5, "grad": True},
        # one token through 8 of 64 experts: a single sequence being decoded
        {"name": "moe_1", "kind": "moe", "T": 1, "H": 4096, "F": 1536, "E": 64, "k": 8, "dtype": "bf16",
         "zipf": False, "pad": 0},
        # a few sequences, float32, sizes that no tile divides
        {"name": "moe_5_odd_f32", "kind": "moe", "T": 5, "H": 1040, "F": 432, "E": 20, "k": 3, "dtype": "f32",
         "zipf": False, "pad": 1},
        # a decode batch with some empty slots
        {"name": "moe_64", "kind": "moe", "T": 64, "H": 4096, "F": 1536, "E": 64, "k": 8, "dtype": "bf16",
         "zipf": False, "pad": 3},
        # the large layer with skewed experts: some get most tokens, many get none
        {"name": "moe_24_large", "kind": "moe", "T": 24, "H": 7168, "F": 2048, "E": 128, "k": 8, "dtype": "bf16",
         "zipf": True, "pad": 0},
        # one token through a dense projection
        {"name": "linear_1", "kind": "linear", "M": 1, "K": 4096, "N": 4096, "dtype": "bf16", "bias": False},
        # a ragged decode batch, with bias
        {"name": "linear_50", "kind": "linear", "M": 50, "K": 7168, "N": 2048, "dtype": "bf16", "bias": True},
        # a prompt of odd length, an odd number of outputs, float32
        {"name": "linear_1001_f32", "kind": "linear", "M": 1001, "K": 1536, "N": 4099, "dtype": "f32", "bias": True},
        # the shared expert over the 16384-token step
        {"name": "mlp_16384", "kind": "mlp", "M": 16384, "H": 4096, "F": 1536, "dtype": "bf16"},
        # the large step's projection
        {"name": "linear_65536", "kind": "linear", "M": 65536, "K": 7168, "N": 2048, "dtype": "bf16", "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["gate", "moe", "moe", "linear", "linear", "mlp"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "gate":
        E = _log(rng, 8, 256)
        return {"kind": kind, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(E, 10)), "dtype": dtype,
                "renorm": rng.random() < 0.5, "masked": rng.choice([0, 0, rng.randint(1, E // 2)]),
                "grad": rng.random() < 0.7}
    if kind == "moe":
        E, T = _log(rng, 8, 128), _log(rng, 1, 128)
        return {"kind": kind, "T": T, "H": 16 * _log(rng, 32, 448), "F": 16 * _log(rng, 16, 128), "E": E,
                "k": rng.randint(1, 8), "dtype": dtype, "zipf": rng.random() < 0.5, "pad": rng.choice([0, 0, T // 4])}
    if kind == "linear":
        while True:
            M, K, N = _log(rng, 1, 65536), 16 * _log(rng, 16, 448), _log(rng, 64, 8192)
            if M * K * N <= 65536 * 7168 * 2048 and M * N <= 65536 * 2048:
                return {"kind": kind, "M": M, "K": K, "N": N, "dtype": dtype, "bias": rng.random() < 0.5}
    # bf16 alone: in float32 the last bit of the SwiGLU decides codes, and with them more than float32 outputs resolve
    return {"kind": kind, "M": _log(rng, 1, 16384), "H": 16 * _log(rng, 16, 256), "F": 16 * _log(rng, 16, 96),
            "dtype": "bf16"}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _outliers(g, x, factor=20.0):
    """0.1% of the entries scaled up, as activations have them."""
    return torch.where(torch.rand(x.shape, generator=g, device=DEV) < 1e-3, x * factor, x)


def _nvfp4_weights(g, E, N, K):
    """N(0, 0.02) weights in NVFP4: codes [E, N, K/2], E4M3 scale bytes [E, N, K/16], outer scales [E]."""
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((E, N, K // 16), dtype=torch.uint8, device=DEV)
    outer = torch.empty((E,), dtype=torch.float32, device=DEV)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for e in range(E):
        w = (_normal(g, N, K) * 0.02).reshape(N, K // 16, 16)
        st = w.abs().amax() / 2688.0
        s8 = (w.abs().amax(-1) / (6.0 * st)).clamp(max=448.0).to(torch.float8_e4m3fn)
        y = w / (s8.float() * st).clamp(min=1e-30).unsqueeze(-1)
        c = (torch.bucketize(y.abs(), edges).to(torch.uint8) + (y < 0).to(torch.uint8) * 8).reshape(N, K // 2, 2)
        codes[e], scales[e], outer[e] = c[..., 0] + c[..., 1] * 16, s8.view(torch.uint8), st
    return codes, scales, outer


def _int8_weights(g, N, K):
    """N(0, 0.02) weights in 8-bit integers with a scale for each output channel."""
    codes = torch.empty((N, K), dtype=torch.int8, device=DEV)
    scales = torch.empty((N,), dtype=torch.float32, device=DEV)
    w = _normal(g, N, K) * 0.02
    scales.copy_(w.abs().amax(1) / 127.0)
    codes.copy_(torch.round(w / scales.unsqueeze(1)).clamp(-127, 127).to(torch.int8))
    return codes, scales


def _logp(c):
    """Log popularity of the experts: even, or Zipf(1.1)."""
    return -1.1 * np.log(np.arange(1, c["E"] + 1)) if c["zipf"] else np.zeros(c["E"])


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["kind"] == "gate":
        x = 2.0 * _normal(g, c["T"], c["E"])
        if c["masked"]:  # experts out of service
            x[:, torch.randperm(c["E"], generator=g, device=DEV)[:c["masked"]]] = -math.inf
        s["logits"] = x.to(_DT[c["dtype"]])
        s["dweights"] = _normal(g, c["T"], c["k"]) * 1e-3
    elif c["kind"] == "moe":
        x = _normal(g, c["T"], c["H"])
        if c["zipf"]:  # the heavy-tailed activations of the skewed workload: Student-t(3)
            x = x / torch.sqrt(sum(_normal(g, c["T"], c["H"]).square() for _ in range(3)) / 3)
        s["x"] = x.to(_DT[c["dtype"]])
        u = torch.rand((c["T"], c["E"]), generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)
        order = torch.tensor(_logp(c), device=DEV, dtype=torch.float32) - torch.log(-torch.log(u))
        ids = torch.argsort(order, dim=1, descending=True)[:, :c["k"]].to(torch.int32)
        w = torch.softmax(_normal(g, c["T"], c["k"]), dim=1)
        if c["pad"]:  # empty slots of the batch
            ids[c["T"] - c["pad"]:] = -1
            w[c["T"] - c["pad"]:] = 0
        s["ids"], s["w"] = ids.contiguous(), w.contiguous()
        s["w13"] = _nvfp4_weights(g, c["E"], 2 * c["F"], c["H"])
        s["w2"] = _nvfp4_weights(g, c["E"], c["H"], c["F"])
    elif c["kind"] == "linear":
        s["x"] = _outliers(g, _normal(g, c["M"], c["K"])).to(_DT[c["dtype"]])
        s["w"] = _int8_weights(g, c["N"], c["K"])
        s["bias"] = _normal(g, c["N"]) * 0.1 if c["bias"] else None
    else:
        s["x"] = _outliers(g, _normal(g, c["M"], c["H"])).to(_DT[c["dtype"]])
        s["w13"] = _int8_weights(g, 2 * c["F"], c["H"])
        s["w2"] = _int8_weights(g, c["H"], c["F"])
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_gate(s):
    c = s["case"]
    x = s["logits"].float()
    E, k = c["E"], c["k"]
    vals, ids = torch.sort(x, dim=1, descending=True, stable=True)  # stable: ties go to the lowest index
    vals, ids = vals[:, :k], ids[:, :k]
    there = vals > -math.inf
    m = torch.where(there[:, :1], vals[:, :1], 0.0)
    p = torch.exp(vals - m)
    total = p.sum(1, keepdim=True) if c["renorm"] else torch.exp(x - m).sum(1, keepdim=True)
    w = p / total.clamp(min=1e-38)
    out = {"weights": w, "ids": torch.where(there, ids, -1).to(torch.int32)}
    if c["grad"]:
        dw = torch.where(there, s["dweights"], 0.0)
        inner = (w * dw).sum(1, keepdim=True)
        if c["renorm"]:
            dx = torch.zeros_like(x).scatter(1, ids, w * (dw - inner))
        else:
            dx = torch.exp(x - m) / total.clamp(min=1e-38) * (torch.zeros_like(x).scatter(1, ids, dw) - inner)
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _decoded(codes, scales, outer):
    """NVFP4 [A, N, K/2], [A, N, K/16], [A] -> float32 [A, N, K]."""
    table = torch.tensor([[_E2M1[b & 15], _E2M1[b >> 4]] for b in range(256)], device=DEV)
    A, N, K2 = codes.shape
    q = table[codes.int()].reshape(A, N, K2 // 8, 16)
    return (q * (scales.view(torch.float8_e4m3fn).float() * outer[:, None, None]).unsqueeze(-1)).reshape(A, N, 2 * K2)


def _plain_moe(s):
    c = s["case"]
    T, k, E, F, H = c["T"], c["k"], c["E"], c["F"], c["H"]
    x, ids = s["x"].float(), s["ids"].long()
    w = torch.where(ids >= 0, s["w"], 0.0).reshape(-1)
    flat = ids.clamp(min=0).reshape(-1)
    token = torch.arange(T, device=DEV).repeat_interleave(k)
    if T * k < E:  # the chosen experts' weights alone
        experts, place = flat, torch.arange(T * k, device=DEV)
    else:
        experts, place = torch.arange(E, device=DEV), flat
    w13 = _decoded(*(t[experts] for t in s["w13"]))
    w2 = _decoded(*(t[experts] for t in s["w2"]))
    A = w13.shape[0]
    h13 = (x @ w13.reshape(A * 2 * F, H).t()).reshape(T, A, 2 * F)[token, place]
    g, u = h13[:, :F], h13[:, F:]
    h = g / (1 + torch.exp(-g)) * u
    z = torch.zeros((A, T, F), device=DEV).index_put((place, token), h * w[:, None], accumulate=True)
    y = torch.zeros((T, H), device=DEV)
    y = y + torch.bmm(z, w2.transpose(1, 2).contiguous()).sum(0)
    return y.to(s["x"].dtype)


def _plain_quantize(x):
    x = x.float()
    a = x.abs().amax(1)
    sc = torch.where(a > 0, a / 127.0, 1.0)
    return torch.round(x * (1.0 / sc).unsqueeze(1)).clamp(-127, 127), sc


def _plain_linear(x, w, sw, bias, dtype):
    q, sx = _plain_quantize(x)
    y = (q @ w.float().t()) * sx.unsqueeze(1) * sw
    return (y if bias is None else y + bias).to(dtype)


def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s)
    if c["kind"] == "gate":
        return _plain_gate(s)
    if c["kind"] == "moe":
        return _plain_moe(s)
    if c["kind"] == "linear":
        return _plain_linear(s["x"], *s["w"], s["bias"], s["x"].dtype)
    h13 = _plain_linear(s["x"], *s["w13"], None, s["x"].dtype).float()
    g, u = h13[:, :c["F"]], h13[:, c["F"]:]
    return _plain_linear(g / (1 + torch.exp(-g)) * u, *s["w2"], None, s["x"].dtype)


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import block_scaled_bit_quantize_amd as bsq
    c = s["case"]
    if c["kind"] == "gate":
        w, ids = bsq.moe_gate(s["logits"], c["k"], renormalize=c["renorm"])
        out = {"weights": w, "ids": ids}
        if c["grad"]:
            out["dlogits"] = bsq.moe_gate_backward(s["dweights"], w, ids, s["logits"], renormalize=c["renorm"])
        return out
    if c["kind"] == "moe":
        return bsq.moe_few_tokens_nvfp4(s["x"], s["ids"], s["w"], *s["w13"], *s["w2"])
    if c["kind"] == "linear":
        return bsq.linear_int8(s["x"], *s["w"], bias=s["bias"], out_dtype=s["x"].dtype)
    x = s["x"]
    h13 = bsq.gemm_int8(*bsq.quantize_int8(x), *s["w13"], out_dtype=x.dtype)
    return bsq.gemm_int8(*bsq.swiglu_quantize_int8(h13), *s["w2"], out_dtype=x.dtype)


# ------------------------------------------------------------------ what a pass cannot do without
def _active(c):
    """Distinct experts that a batch of the case's routing reaches, from draws of a fixed seed."""
    T = c["T"] - c["pad"]
    got = []
    for k in range(8):
        u = np.random.default_rng(k).random((T, c["E"])).clip(1e-9, 1 - 1e-9)
        order = np.argsort(-(_logp(c) - np.log(-np.log(u))), axis=1)[:, :c["k"]]
        got.append(len(np.unique(order)))
    return sum(got) / len(got)


def work(case):
    c = case
    sz = _SIZE[c["dtype"]]
    if c["kind"] == "gate":
        T, E, k = c["T"], c["E"], c["k"]
        b = T * E * sz + T * k * 8
        if c["grad"]:
            b += T * k * 4 + T * E * sz
        return {"bytes": b, "flops": T * E * 8}
    if c["kind"] == "moe":
        T, H, F, k = c["T"], c["H"], c["F"], c["k"]
        return {"bytes": _active(c) * 3 * F * H * 0.5625 + 2 * T * H * sz + T * k * 8,
                "flops": 6 * (T - c["pad"]) * k * F * H}
    if c["kind"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": M * K * sz + N * K + 4 * N + M * N * sz, "flops": 2 * M * K * N}
    M, H, F = c["M"], c["H"], c["F"]
    return {"bytes": 2 * M * H * sz + 3 * H * F, "flops": 6 * M * H * F}


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_gate(s):
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    T, E, k = c["T"], c["E"], c["k"]
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k]
    l = np.take_along_axis(x, ids, 1)
    ok = np.isfinite(l)
    top = np.where(ok[:, :1], l[:, :1], 0.0)
    ex = np.exp(x - top)  # zero where masked
    e = np.where(ok, np.exp(np.where(ok, l, 0) - top), 0)
    den = e.sum(1, keepdims=True) if c["renorm"] else ex.sum(1, keepdims=True)
    den = np.where(den > 0, den, 1.0)
    w = e / den
    out = {"weights": torch.from_numpy(w), "ids": None}
    if c["grad"]:
        dw = s["dweights"].double().cpu().numpy() * ok
        # d w_j / d l_i = w_j ([i = j] - p_i), p over the experts that share the denominator
        p = np.zeros((T, E))
        if c["renorm"]:
            np.put_along_axis(p, ids, w, 1)
        else:
            p = ex / den
        d = -p * (w * dw).sum(1, keepdims=True)
        np.put_along_axis(d, ids, np.take_along_axis(d, ids, 1) + w * dw, 1)
        out["dlogits"] = torch.from_numpy(d)
    return out


def _exact_weights(parts, e):
    codes, scales, outer = (t[e] for t in parts)
    c = codes.long()
    nib = torch.stack([c & 15, c >> 4], -1).flatten(1)
    mag = nib & 7
    ex, m = mag >> 1, mag & 1  # two exponent bits of bias 1, one mantissa bit
    v = torch.where(ex == 0, m.double() * 0.5, (1 + m.double() / 2) * torch.exp2((ex - 1).double()))
    v = torch.where(nib >= 8, -v, v)
    b = scales.long()
    be, bm = (b >> 3) & 15, b & 7
    sv = torch.where(be == 0, bm.double() * 2.0 ** -9, (1 + bm.double() / 8) * torch.exp2((be - 7).double()))
    return v * sv.repeat_interleave(16, 1) * outer.double()


def _exact_moe(s):
    c = s["case"]
    x, ids, w = s["x"].double(), s["ids"].cpu().numpy(), s["w"].double()
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    for e in np.unique(ids[ids >= 0]):
        t, j = (torch.from_numpy(v).to(DEV) for v in np.nonzero(ids == e))
        h = x[t] @ _exact_weights(s["w13"], int(e)).t()
        a = h[:, :c["F"]] * torch.sigmoid(h[:, :c["F"]]) * h[:, c["F"]:]
        y.index_add_(0, t, (a @ _exact_weights(s["w2"], int(e)).t()) * w[t, j][:, None])
    return y


def _exact_linear(x, w, sw, bias):
    x = x.double()
    out = torch.empty((x.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    wt = w.double().t().contiguous()
    for r in range(0, x.shape[0], 8192):
        v = x[r:r + 8192]
        sc = v.abs().amax(1, keepdim=True) / 127
        sc = torch.where(sc == 0, torch.ones_like(sc), sc)
        out[r:r + 8192] = (torch.clamp(torch.round(v / sc), -127, 127) @ wt) * sc * sw.double()
    return out if bias is None else out + bias.double()


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["kind"] == "gate":
        return _exact_gate(s)
    if c["kind"] == "moe":
        return _exact_moe(s)
    if c["kind"] == "linear":
        return _exact_linear(s["x"], *s["w"], s["bias"])
    h = _exact_linear(s["x"], *s["w13"], None).to(s["x"].dtype).double()
    return _exact_linear(h[:, :c["F"]] * torch.sigmoid(h[:, :c["F"]]) * h[:, c["F"]:], *s["w2"], None)
