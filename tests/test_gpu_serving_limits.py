"""The router and the 8-bit products past the sizes of one launch (2^32
work-items along a grid's dimension). The inputs repeat a block of rows whose
number is coprime to the launches' slices, so every block of the output has to
hold the same bits as the block alone."""
import pytest
import torch

import block_scaled_bit_quantize_amd as bsq
from _gpu_util import DEV, log

pytestmark = pytest.mark.gpu

P = 1009  # rows of the repeated block


def blocks(rows, period=P):
    return rows // period + 1


def same(out, one, period=P, step=4096):
    """Every block of `out`'s rows equals `one`; a part at a time, to bound the memory."""
    out = out.view(-1, period, *one.shape[1:])
    return all(bool((out[i:i + step] == one).all()) for i in range(0, out.shape[0], step))


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,E,k,rows", [(torch.float32, 8, 1, 1 << 28), (torch.bfloat16, 257, 2, 1 << 26)])
def test_gate_past_one_launch(dtype, E, k, rows):
    m = blocks(rows)
    log(f"gate past one launch {m * P} x {E}")
    one = torch.randn((P, E), device=DEV).to(dtype)
    x = one.repeat(m, 1)
    for renorm in (True, False):
        w1, i1 = bsq.moe_gate(one, k, renormalize=renorm)
        w, i = bsq.moe_gate(x, k, renormalize=renorm)
        assert same(i, i1) and same(w, w1)
        d1 = bsq.moe_gate_backward(w1, w1, i1, one, renormalize=renorm)
        d = bsq.moe_gate_backward(w, w, i, x, renormalize=renorm)
        assert same(d, d1)
        del w, i, d


@pytest.mark.parametrize("C,rows", [(16, 1 << 26)])
def test_quantize_int8_past_one_launch(C, rows):
    m = blocks(rows)
    log(f"quantize_int8 past one launch {m * P} x {C}")
    one = torch.randn((P, C), device=DEV).bfloat16()
    q1, s1 = bsq.quantize_int8(one)
    x = one.repeat(m, 1)
    q, s = bsq.quantize_int8(x)
    assert same(q, q1) and same(s, s1)
    del q, s, x
    one = torch.randn((P, 2 * C), device=DEV).bfloat16()
    q1, s1 = bsq.swiglu_quantize_int8(one)
    q, s = bsq.swiglu_quantize_int8(one.repeat(m, 1))
    assert same(q, q1) and same(s, s1)


@pytest.mark.parametrize("M,N,call", [(2, 1 << 28, "gemm"), (1, 1 << 27, "linear")])
def test_few_rows_of_more_channels_than_one_launch(M, N, call):
    m = blocks(N)
    log(f"{call}_int8 past one launch {M} x {m * P}")
    b1 = torch.randint(-127, 128, (P, 16), device=DEV, dtype=torch.int8)
    s1 = torch.rand(P, device=DEV)
    bias1 = torch.rand(P, device=DEV)
    x = torch.randn((M, 16), device=DEV)
    run = (lambda *w, bias: bsq.gemm_int8(*bsq.quantize_int8(x), *w, bias=bias)) if call == "gemm" else \
        (lambda *w, bias: bsq.linear_int8(x, *w, bias=bias))
    y1 = run(b1, s1, bias=bias1)
    y = run(b1.repeat(m, 1), s1.repeat(m), bias=bias1.repeat(m))
    for r in range(M):
        assert same(y[r], y1[r])


def test_more_rows_than_one_launch_of_tiles():
    period = 2387                      # divides 2^31 - 2, which is more than 2^24 - 1 tiles of 128 rows
    m = ((1 << 31) - 2) // period
    assert m * period == (1 << 31) - 2
    log(f"gemm_int8 past one launch {m * period} x 1")
    a1 = torch.randint(-127, 128, (period, 16), device=DEV, dtype=torch.int8)
    s1 = torch.rand(period, device=DEV)
    b, sb = torch.randint(-127, 128, (1, 16), device=DEV, dtype=torch.int8), torch.rand(1, device=DEV)
    y1 = bsq.gemm_int8(a1, s1, b, sb)
    y = bsq.gemm_int8(a1.repeat(m, 1), s1.repeat(m), b, sb)
    assert same(y, y1, period)
