"""Token log probabilities, entropies, alternatives and gradients against the 64-bit oracle.

Bounds. e^z is off by (2 + 1.5 |z|) 2^-24, and |z| e^z is at most e^-1, so that a sum of V terms is off by 2^-24 of
itself times 2 + 1.5 |log p| where its weight lies, plus one rounding for each addition in a thread (V / 256 + 32 of
them, and at most V); the logarithm's error is the sum's relative one; differences add half a step of their size. An
entropy is a sum of p |log p|, off by the same factor times (1 + H). Alternatives' ids are exact."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log
from oracle import logprob as L

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
OUT_EPS = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def dev(a, dtype=F32):
    x = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)
    return x, x.float().cpu().numpy().astype(np.float64)


def relative(V, entropy):
    adds = min(V, V / 256 + 32 + 16)
    return (adds + 8 + 1.5 * (entropy + 1)) * 2.0 ** -24


def check(x, targets, top, dtype, seed=5):
    T, V = x.shape
    log(f"token_logprobs {T} x {V} top {top} {dtype}")
    xd, xv = dev(x, dtype)
    td = torch.from_numpy(np.asarray(targets, dtype=np.int64)).to(DEV)
    lp, entropy, stats, tl, ti = bsq.token_logprobs(xd, td, top=top)
    assert lp.shape == entropy.shape == (T,) and stats.shape == (T, 2)
    wl, we, wt, wi = L.token_logprobs(xv, np.asarray(targets), top)
    rel = relative(V, we)
    size = np.where(np.isfinite(wl), np.abs(wl), 0.0)
    sized = np.abs(np.where(xv > -np.inf, xv, 0.0)).max(1)  # differences of logits of this size
    tol = rel + 4 * 2.0 ** -24 * (size + 1)
    same = h(lp) == wl  # minus infinity for a masked target
    off = np.abs(np.where(same, 0.0, h(lp)) - np.where(same, 0.0, wl))
    assert (off <= tol).all(), float((off / tol).max())
    assert (np.abs(h(entropy) - we) <= 2 * rel * (1 + we) + 4 * 2.0 ** -24 * (1 + we)).all()
    lse = h(stats.double().sum(1))
    some = (xv > -np.inf).any(1)
    want = np.where(some, np.log(np.exp(xv - np.where(some, xv.max(1), 0.0)[:, None]).sum(1).clip(1e-300)) + np.where(some, xv.max(1), 0), 0)
    assert (np.abs(lse - want) <= rel + 2.0 ** -23 * (np.abs(want) + sized)).all()
    if top:
        np.testing.assert_array_equal(h(ti), wi)
        got = h(tl).astype(np.float64)
        fine = np.isfinite(wt)
        assert (got[~fine] == -np.inf).all()
        tt = rel[:, None] + 4 * 2.0 ** -24 * (1 + np.abs(np.where(fine, wt, 0)))
        assert (np.abs(np.where(fine, got, 0) - np.where(fine, wt, 0)) <= tt).all()
    else:
        assert tl is None and ti is None
    rng = np.random.default_rng(seed)
    g, e = rng.standard_normal(T).astype(np.float32), rng.standard_normal(T).astype(np.float32)
    gd, ed = torch.from_numpy(g).to(DEV), torch.from_numpy(e).to(DEV)
    logp = np.where(xv > -np.inf, L.log_softmax(xv), 0.0)
    for a, b in ((gd, ed), (gd, None), (None, ed)):
        d = bsq.token_logprobs_backward(a, b, xd, td, stats, entropy)
        assert d.dtype == dtype and d.shape == xd.shape
        ga, eb = (g if a is not None else 0 * g), (e if b is not None else 0 * e)
        do = L.gradient(ga, eb, xv, np.asarray(targets))
        # p (|g| + |h| (|log p| + H)), p's exponent off by the log-sum-exp's error and |log p| 2^-23
        big = np.abs(ga)[:, None] + np.abs(eb)[:, None] * (np.abs(logp) + we[:, None] + 1)
        off = (4 * rel[:, None] + 2.0 ** -21 * (1 + np.abs(logp))) * np.exp(np.minimum(logp, 0)) * big
        # the exponential instruction gives 0 for a p below 2^-126: all of p times the rest is then missing
        tiny = 2.0 ** -126 * big + 2.0 ** -149
        dd = d.double().cpu().numpy()
        tol = off + OUT_EPS[dtype] * (np.abs(do) + off) + 2.0 ** -24 * np.abs(ga)[:, None] * (np.abs(do) > 0) + tiny
        assert (np.abs(dd - do) <= tol).all(), float((np.abs(dd - do) / tol).max())
        assert (dd[xv == -np.inf] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,V,top", [(1, 1, 1), (3, 2, 2), (1, 64, 64), (5, 63, 20), (4, 129, 5), (7, 1000, 64), (2, 4096, 1),
                                     (3, 4097, 64), (1, 100003, 20), (9, 32000, 5), (64, 2051, 3), (2, 131072, 64), (33, 517, 0),
                                     (1, 50021, 0), (1, 300001, 40), (1, 1 << 20, 64), (1, (1 << 20) - 3, 7)])
def test_shapes(T, V, top, dtype):
    rng = np.random.default_rng(T + V)
    x = rng.standard_normal((T, V)) * 3
    t = rng.integers(0, V, T)
    if T > 2:
        t[1], t[2] = -100, V
    check(x, t, top, dtype)
    x[rng.random((T, V)) < 0.7] = -np.inf
    check(x, t, top, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,V,top", [(1030, 257, 0), (1030, 130, 9), (2000, 4099, 0), (300, 33001, 12)])
def test_many_rows(T, V, top, dtype):
    rng = np.random.default_rng(T + V)
    check(rng.standard_normal((T, V)) * 3, rng.integers(-1, V, T), top, dtype)


@pytest.mark.parametrize("V", [100, 5000, 40000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_special_rows(V, dtype):
    low = float(torch.finfo(F32).min)
    x = np.zeros((10, V))
    x[0] = -np.inf                          # nothing left
    x[1] = -np.inf
    x[1, V - 1] = 5.0                       # one left
    x[2] = low if dtype == F32 else -3e38   # lowest finite values: no masks
    x[3] = np.where(np.arange(V) % 2, 0.0, -0.0)
    x[4] = 1000.0                           # all tie
    x[5] = np.arange(V) * 0.5               # the maximum rises all along
    x[6] = -np.arange(V) * 0.5              # and falls
    x[7, V // 2] = 300.0                    # one takes all
    x[8, :V // 2] = -np.inf                 # the first parts of the row are empty
    x[9, ::64] = 2.0                        # blocks that tie
    t = np.array([0, 0, 1, 2, V - 1, V - 1, 0, V // 2, V - 1, 64])
    check(x, t, 40, dtype)
    check(x, t, 0, dtype)


def test_alternatives_in_one_block():
    """All of the alternatives next to each other, at places that cross blocks, and many equal ones."""
    rng = np.random.default_rng(2)
    for V in (1500, 70001):
        x = rng.standard_normal((40, V))
        for r in range(40):
            at = rng.integers(0, V - 64)
            x[r, at:at + 64] = 10 + rng.integers(0, 5, 64)
        check(x, rng.integers(0, V, 40), 64, BF16)
        check(x, rng.integers(0, V, 40), 33, F32)


@pytest.mark.parametrize("V", [77, 9001])
def test_nan_and_infinite_rows(V):
    x = torch.randn((6, V), device=DEV)
    clean = x.clone()
    x[1, V // 2] = float("nan")
    x[3, 5] = float("inf")
    t = torch.full((6,), 3, dtype=torch.int64, device=DEV)
    g = torch.ones(6, device=DEV)
    lp, entropy, stats, tl, ti = bsq.token_logprobs(x, t, top=4)
    d = bsq.token_logprobs_backward(g, g, x, t, stats, entropy)
    want = bsq.token_logprobs(clean, t, top=4)
    dw = bsq.token_logprobs_backward(g, g, clean, t, want[2], want[1])
    keep = [0, 2, 4, 5]
    for a, b in zip((lp, entropy, stats, tl, ti, d), (*want, dw)):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(lp[[1, 3]]).all() and torch.isnan(entropy[[1, 3]]).all() and torch.isnan(d[[1, 3]]).any(1).all()
    assert ((ti >= 0) & (ti < V)).all() and (ti[3, 0] == 5) and not (ti[1] == V // 2).any()


def test_large():
    """Offsets past 2^31 elements: the last rows against the same rows by themselves."""
    T, V = 2100, (1 << 20) - 1
    log("token_logprobs large")
    x = torch.empty((T, V), dtype=BF16, device=DEV)
    x[:] = torch.randn((1, V), device=DEV).to(BF16)
    x[-3:] = torch.randn((3, V), device=DEV).to(BF16) * 2
    t = torch.arange(T, device=DEV)
    g = torch.randn(T, device=DEV)
    out = bsq.token_logprobs(x, t, top=3)
    d = bsq.token_logprobs_backward(g, g, x, t, out[2], out[1])
    last = x[-3:].clone()
    alone = bsq.token_logprobs(last, t[-3:].contiguous(), top=3)
    for a, b in zip(out[:4], alone[:4]):
        # cut into parts for more workgroups: other orders of the same sums
        assert torch.allclose(a[-3:], b, rtol=relative(V, 14.0) * 2, atol=relative(V, 14.0) * 2)
    assert torch.equal(out[4][-3:], alone[4])
    da = bsq.token_logprobs_backward(g[-3:].contiguous(), g[-3:].contiguous(), last, t[-3:].contiguous(),
                                     out[2][-3:].contiguous(), out[1][-3:].contiguous())
    assert torch.equal(d[-3:], da)


def test_empty_and_refusals():
    x = torch.zeros((0, 9), device=DEV)
    t = torch.zeros(0, dtype=torch.int64, device=DEV)
    out = bsq.token_logprobs(x, t, top=2)
    assert out[0].shape == (0,) and out[3].shape == (0, 2)
    assert bsq.token_logprobs_backward(out[0], None, x, t, out[2], out[1]).shape == (0, 9)
    x = torch.zeros((4, 9), device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    for bad in ((x.half(), t), (x, t.int()), (x, t[:3]), (x[0], t), (x.t(), t), (x, t.cpu())):
        with pytest.raises(bsq.BsqError):
            bsq.token_logprobs(*bad)
    for top in (-1, 10, 65):
        with pytest.raises(bsq.BsqError):
            bsq.token_logprobs(x, t, top=top)
    lp, e, s, _, _ = bsq.token_logprobs(x, t)
    for bad in ((None, None, x, t, s, e), (lp.double(), None, x, t, s, e), (lp, e[:2], x, t, s, e), (lp, None, x, t, s[:, :1], e),
                (lp, None, x, t.int(), s, e), (lp, None, x, t, s, e[:3])):
        with pytest.raises(bsq.BsqError):
            bsq.token_logprobs_backward(*bad)


@pytest.mark.parametrize("T,V,top", [(3, 50001, 7), (1500, 600, 0)])
def test_stream_and_graph(T, V, top):
    x = torch.randn((T, V), device=DEV)
    t = torch.randint(0, V, (T,), device=DEV)
    g = torch.randn(T, device=DEV)

    def step():
        out = bsq.token_logprobs(x, t, top=top)
        return [v for v in out if v is not None] + [bsq.token_logprobs_backward(g, g, x, t, out[2], out[1])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step()
    torch.cuda.current_stream().wait_stream(s)
    for i in range(4):
        x.copy_(torch.randn((T, V), device=DEV) * (1 + i))
        t.copy_(torch.randint(0, V, (T,), device=DEV))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
