"""The grouped router against its 64-bit oracle: the selection exactly, weights and
gradients within bounds.

Bounds. An exponential is off by 2^-22 (its instruction 2^-23, the carried
rounding and one rounding more), and by 2^-24 of its argument where that is a
difference; a weight has two of them, their sum and quotient, a sum of k terms
and two more roundings: (32 + k + span) 2^-24 relative, span the largest
difference of logits that enters. A gradient is a product of such factors, each
within [0, scale], and of a difference of incoming gradients."""
import numpy as np
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, h, log, t
from oracle import router as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
OUT_EPS = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def dev(a, dtype=F32):
    x = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)
    return x, x.float().cpu().numpy().astype(np.float64)


def check(x, k, dtype, bias=None, groups=1, group_k=None, group_top=2, score="sigmoid", renorm=True, scale=1.0):
    log(f"group_gate {x.shape} k {k} {dtype} groups {groups} {group_k} {group_top} {score} {renorm} {scale} "
        f"bias {bias is not None}")
    xd, xv = dev(x, dtype)
    b = None if bias is None else np.asarray(bias, dtype=np.float32)
    w, ids = bsq.moe_gate_grouped(xd, k, bias=None if b is None else t(b), groups=groups, group_k=group_k,
                                  group_top=group_top, score=score, renormalize=renorm, scale=scale)
    assert w.shape == ids.shape == (x.shape[0], k) and w.dtype == F32 and ids.dtype == torch.int32
    wo, io = R.group_gate(xv, k, b, groups, group_k, group_top, score, renorm, scale)
    np.testing.assert_array_equal(h(ids), io)
    finite = xv[np.isfinite(xv)]
    span = 2 * min(float(np.abs(finite).max()) if finite.size else 0.0, 256.0)
    rel = (32 + x.shape[1] + span) * 2.0 ** -24
    # exponentials below the normal range may be 0
    np.testing.assert_allclose(h(w), wo, rtol=rel, atol=scale * 2.0 ** -120)
    g = np.random.default_rng(5).standard_normal(w.shape).astype(np.float32)
    d = bsq.moe_gate_grouped_backward(t(g), w, ids, xd, score=score, renormalize=renorm, scale=scale)
    assert d.dtype == dtype and d.shape == xd.shape
    do = R.group_gate_grad(g, io, xv, score, renorm, scale)
    size = scale * np.abs(g).max(1, keepdims=True)
    tol = 4 * (rel + k * 2.0 ** -24) * size + OUT_EPS[dtype] * np.abs(do)
    assert (np.abs(d.double().cpu().numpy() - do) <= tol).all()
    return h(ids)


SHAPES = [  # T, E, k, groups, group_k
    (1, 64, 8, 8, 4), (37, 64, 8, 8, 4), (130, 128, 8, 8, 4), (33, 256, 8, 8, 4), (9, 256, 16, 4, 2), (5, 128, 6, 2, 1),
    (7, 64, 3, 16, 5), (6, 128, 4, 32, 3), (5, 256, 15, 64, 20), (17, 60, 6, 5, 3), (4, 63, 9, 7, 2), (3, 96, 64, 3, 2),
    (21, 32, 4, 4, 2), (8, 16, 2, 16, 2), (3, 1024, 64, 64, 9), (2, 1000, 8, 8, 3), (5, 300, 63, 3, 1), (3, 1, 1, 1, 1),
    (4, 2, 1, 2, 1), (66, 128, 8, 1, 1), (9, 20, 20, 1, 1), (3, 512, 5, 1, 1),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,group_k", SHAPES)
def test_shapes(T, E, k, groups, group_k, score, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    x = rng.standard_normal((T, E)) * 2
    bias = rng.standard_normal(E) * (0.1 if score == "sigmoid" else 0.5 / E)
    check(x, k, dtype, bias, groups, group_k, 2, score, True, 2.5)
    check(x, k, dtype, None, groups, group_k, 1, score, False)
    x[rng.random((T, E)) < 0.6] = -np.inf
    check(x, k, dtype, bias, groups, group_k, 1, score, True)
    check(x, k, dtype, bias, groups, group_k, 2, score, False, 0.5)


@pytest.mark.parametrize("E,groups", [(64, 8), (60, 5), (512, 8), (128, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_special_rows(E, groups, score):
    low = float(torch.finfo(F32).min)
    rows = np.zeros((10, E))
    rows[0] = -np.inf                                # nothing left
    rows[1] = -np.inf
    rows[1, E - 1] = 3.0                             # one left
    rows[2] = low                                    # lowest finite value: not a mask
    rows[3] = np.where(np.arange(E) % 2, 0.0, -0.0)  # both zeros tie
    rows[4] = 7.0                                    # all tie
    rows[5] = np.nan
    rows[6, 1::2] = np.nan                           # NaN masks its expert only
    rows[7] = low
    rows[7, 5] = 100.0
    rows[8] = np.arange(E) % 3 * 40.0                # float64 sigmoids of 40 and 80 are both 1
    rows[9] = -np.inf
    rows[9, E // groups:2 * (E // groups)] = 1.0     # all that is left in one group
    for group_top in (1, 2):
        for renorm in (True, False):
            check(rows, 4, F32, None, groups, max(1, groups // 2), group_top, score, renorm)
    bias = np.zeros(E)
    bias[0], bias[1], bias[2] = -np.inf, np.nan, 1e30
    ids = check(rows, 4, F32, bias, groups, max(1, groups // 2), 2, score, True)
    assert not np.isin(ids, (0, 1)).any()
    bias[3] = bias[7] = np.inf
    check(rows, 4, F32, bias, groups, max(1, groups // 2), 1, score, True)


@pytest.mark.parametrize("E,groups", [(64, 8), (64, 4), (60, 5), (256, 8), (512, 8)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_special_biases(E, groups, score):
    """A bias of NaN counts as no key in its group's worth; infinite and huge ones order the groups like others."""
    size = E // groups
    x = np.random.default_rng(E).standard_normal((9, E))
    bias = np.zeros(E)
    bias[:size], bias[size:2 * size] = np.nan, -np.inf
    bias[3], bias[size + 1] = 0.8, 0.7                # the only keys of the first two groups
    bias[2 * size:2 * size + 2] = 0.6                 # two that are worth more together
    for group_top in (1, 2):
        check(x, 2, F32, bias, groups, 1, group_top, score, True)
        check(x, 3, F32, bias, groups, 2, group_top, score, True)
    bias = np.zeros(E)
    bias[1::size] = np.inf                            # one in each group: ties
    check(x, 4, F32, bias, groups, 2, 2, score, True)
    bias[1::2 * size] = 0.0                           # in every second group
    check(x, 4, F32, bias, groups, 1, 2, score, True)
    check(x, 4, F32, bias, groups, 1, 1, score, True)
    most = float(torch.finfo(F32).max)
    bias = np.zeros(E)
    bias[2 * size], bias[2 * size + 1] = most, most / 2  # sums past float32, in two groups
    bias[size:size + 2] = most
    check(x, 3, F32, bias, groups, 1, 2, score, True)
    check(x, min(size + 2, 64), F32, bias, groups, 2, 2, score, True)
    bias = np.full(E, -most)
    bias[3 * size:3 * size + 2] = -most / 2
    check(x, 3, F32, bias, groups, 2, 2, score, True)


@pytest.mark.parametrize("E,groups", [(64, 8), (60, 5), (128, 1), (256, 8), (512, 1), (20, 1)])
def test_infinite_logits(E, groups):
    """+inf in a softmax row: its ids are in range and no expert comes twice; other rows are as ever. Sigmoid rows take
    +inf as a score of 1."""
    x = np.random.default_rng(E).standard_normal((11, E)).astype(np.float32)
    check(x, 4, F32, None, groups, max(1, groups // 2), 2, "sigmoid", False)
    for r in (0, 3, 4):
        x[r, np.arange(r + 1) * 4 + 1] = np.inf
    y = x.copy()
    y[7, 2] = np.inf
    y[7, 3] = -np.inf
    for rows in (x, y):
        for bias in (None, np.linspace(0, 1, E).astype(np.float32)):
            how = dict(groups=groups, group_k=max(1, groups // 2))
            b = None if bias is None else t(bias)
            w, ids = bsq.moe_gate_grouped(t(rows), 4, bias=b, score="softmax", **how)
            wo, io = R.group_gate(rows, 4, bias, groups, how["group_k"], 2, "softmax")
            ids = h(ids)
            assert ((ids >= -1) & (ids < E)).all()
            for r in range(11):
                there = ids[r][ids[r] >= 0]
                assert len(set(there.tolist())) == len(there)
                if np.isfinite(rows[r]).all():
                    np.testing.assert_array_equal(ids[r], io[r])
            check(rows, 4, F32, bias, groups, how["group_k"], 2, "sigmoid", False)


@pytest.mark.parametrize("E,groups,group_k", [(64, 1, 1), (64, 8, 4), (60, 5, 2), (256, 8, 4), (512, 4, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_near_ties(E, groups, group_k, score):
    """Keys that float32 cannot tell apart: neighbouring floats as logits, and biases that make up for the scores'
    differences but for 1e-9 of them."""
    rng = np.random.default_rng(E)
    x = np.full((48, E), 1.0, dtype=np.float32)
    x += rng.integers(0, 4, x.shape).astype(np.float32) * np.float32(2.0 ** -23)
    check(x, 8 if group_k * (E // groups) >= 8 else 4, F32, None, groups, group_k, 2, score, True)
    x[:, ::3] = 20.0 + rng.integers(0, 3, x[:, ::3].shape)  # sigmoids within 2e-9 of 1
    check(x, 8, F32, None, groups, group_k, 1, score, True)
    y = rng.standard_normal((1, E)).astype(np.float32).repeat(40, 0)
    s = R.scores(y[:1].astype(np.float64), score)[0]
    bias = (0.75 - s).astype(np.float32)  # every key is 0.75 but for the bias's rounding
    check(y, 8, F32, bias, groups, group_k, 2, score, False)


def test_bf16_ties_at_the_cut():
    """Equal logits around the last selected one, with a nearly equal key behind them."""
    x = np.full((64, 128), -3.0, dtype=np.float32)
    x[:, 5], x[:, 9] = 3.0, 2.0
    for r in range(64):
        x[r, np.random.default_rng(r).permutation(np.arange(10, 128))[:40]] = 1.0
    check(x, 8, BF16, None)
    s = 1 / (1 + np.exp(-1.0))
    bias = np.zeros(128, dtype=np.float32)
    bias[100] = np.float32(s - 1 / (1 + np.exp(3.0)))  # expert 100's key is as large as the tied ones' but for 1e-8
    check(x, 8, BF16, bias)


@pytest.mark.parametrize("T", [16381, 65536])
def test_many_tokens(T):
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, 128)) * 2
    check(x, 8, BF16, rng.standard_normal(128) * 0.05, 8, 4, 2, "sigmoid", True, 2.5)


def test_gradient_by_differences():
    """The kernels' own weights, differenced: float32 weights of about 0.3 resolve 2^-25, over a step of 2^-7."""
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((4, 24)).astype(np.float32)).to(DEV)
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            how = dict(score=score, renormalize=renorm)
            sel = dict(groups=4, group_k=2, bias=torch.zeros(24, device=DEV), **how)
            w, ids = bsq.moe_gate_grouped(x, 5, **sel)
            g = torch.from_numpy(rng.standard_normal((4, 5)).astype(np.float32)).to(DEV)
            d = bsq.moe_gate_grouped_backward(g, w, ids, x, **how).double().cpu()
            step = 2.0 ** -7
            for e in range(24):
                side = []
                for sign in (1, -1):
                    y = x.clone()
                    y[:, e] += sign * step
                    wy, iy = bsq.moe_gate_grouped(y, 5, **sel)
                    at = torch.where(iy.unsqueeze(1) == ids.unsqueeze(2), wy.unsqueeze(1), 0.0).sum(2)
                    side.append(((g * at).double().sum(1).cpu(), (iy.sort(1).values == ids.sort(1).values).all(1).cpu()))
                same = side[0][1] & side[1][1]  # the selection is held fixed
                diff = (side[0][0] - side[1][0]) / (2 * step)
                # 5 terms of |g| <= 3.5, each off by (32 + 24 + 8) 2^-24 w; third derivatives below 1, times step^2 / 6
                tol = 5 * 3.5 * 64 * 2.0 ** -24 / step + 5 * 3.5 * step ** 2 / 6
                assert ((diff - d[:, e]).abs()[same] <= tol).all()


def test_no_tokens_and_refusals():
    x = torch.zeros((0, 64), device=DEV)
    w, ids = bsq.moe_gate_grouped(x, 8, groups=8, group_k=4)
    assert w.shape == ids.shape == (0, 8)
    assert bsq.moe_gate_grouped_backward(w, w, ids, x).shape == (0, 64)
    x = torch.zeros((4, 64), device=DEV)
    for bad in (dict(k=0), dict(k=65), dict(k=8, groups=7), dict(k=9, groups=8, group_k=1), dict(k=8, groups=8, group_k=9),
                dict(k=8, groups=8, group_k=0), dict(k=8, group_top=3), dict(k=8, score="tanh"), dict(k=8, scale=0.0),
                dict(k=8, scale=float("nan")), dict(k=8, bias=torch.zeros(63, device=DEV)),
                dict(k=8, bias=torch.zeros(64, device=DEV, dtype=BF16)), dict(k=8, bias=torch.zeros(64))):
        with pytest.raises(bsq.BsqError):
            bsq.moe_gate_grouped(x, **bad)
    with pytest.raises(bsq.BsqError):
        bsq.moe_gate_grouped(x.half(), 8)
    with pytest.raises(bsq.BsqError):
        bsq.moe_gate_grouped(x.t(), 2)
    w, ids = bsq.moe_gate_grouped(x, 8)
    for bad in ((w[:, :4], w, ids, x), (w, w, ids.long(), x), (w.double(), w, ids, x), (w, w, ids[:2], x)):
        with pytest.raises(bsq.BsqError):
            bsq.moe_gate_grouped_backward(*bad)


def test_ids_out_of_range_add_nothing():
    x = torch.randn((3, 64), device=DEV)
    w, ids = bsq.moe_gate_grouped(x, 4)
    g = torch.ones_like(w)
    bad = ids.clone()
    bad[:, 3] = torch.tensor([64, -7, 1 << 30], dtype=torch.int32)
    d = bsq.moe_gate_grouped_backward(g, w, bad, x, renormalize=False)
    want = bsq.moe_gate_grouped_backward(g[:, :3].contiguous(), w[:, :3].contiguous(), ids[:, :3].contiguous(), x,
                                         renormalize=False)
    assert torch.equal(d, want)


def test_stream_and_graph():
    x = torch.randn((257, 128), device=DEV)
    g = torch.randn((257, 8), device=DEV)
    bias = torch.randn(128, device=DEV) * 0.1
    how = dict(bias=bias, groups=8, group_k=4)

    def step():
        w, ids = bsq.moe_gate_grouped(x, 8, **how)
        return w, ids, bsq.moe_gate_grouped_backward(g, w, ids, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step()
    torch.cuda.current_stream().wait_stream(s)
    for i in range(4):
        x.copy_(torch.randn((257, 128), device=DEV) * (1 + i))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
