"""Argument checks of the grouped router, the 4-bit groups and the token log probabilities, on the host before any HIP
call (no GPU needed)."""
import os

import pytest

from block_scaled_bit_quantize_amd import _lib

OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE, E_ENUM, E_WORKSPACE, E_LAUNCH = range(8)
FAKE = 0x10000  # a 16-byte aligned non-null value; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.library_path()):
        from block_scaled_bit_quantize_amd.build import build
        build()
    return _lib.load_library()


def caller(fn, base):
    def call(**kw):
        a = list(base)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return fn(*a)
    return call


def test_group_gate(lib):
    # logits, dtype, bias, tokens, E, k, groups, group_k, group_top, score, renorm, scale, weights, ids, stream
    c = caller(lib.bsq_moe_gate_grouped, [FAKE, 0, None, 4, 64, 8, 8, 4, 2, 0, 1, 1.0, FAKE, FAKE, None])
    assert c(a1=2) == E_DTYPE
    for kw in (dict(a8=0), dict(a8=3), dict(a9=2), dict(a10=2), dict(a11=0.0), dict(a11=-1.0), dict(a11=float("nan")),
               dict(a11=float("inf")), dict(a11=2.0 ** 65)):
        assert c(**kw) == E_ENUM, kw
    for kw in (dict(a3=-1), dict(a3=1 << 31), dict(a4=0), dict(a4=1025), dict(a5=0), dict(a5=65), dict(a5=33), dict(a6=0),
               dict(a6=7), dict(a6=65, a4=650), dict(a7=0), dict(a7=9), dict(a6=8, a7=1, a5=9)):
        assert c(**kw) == E_SHAPE, kw
    for i in (0, 12, 13):
        assert c(**{f"a{i}": None}) == E_NULL, i
    for kw in (dict(a0=FAKE + 8), dict(a2=FAKE + 2), dict(a12=FAKE + 1), dict(a13=FAKE + 2)):
        assert c(**kw) == E_ALIGN, kw
    assert c(a3=0, a0=None) == OK
    # dweights, weights, ids, logits, dtype, tokens, E, k, score, renorm, scale, dlogits, stream
    b = caller(lib.bsq_moe_gate_grouped_backward, [FAKE, FAKE, FAKE, FAKE, 1, 4, 64, 8, 1, 0, 1.0, FAKE, None])
    assert b(a4=3) == E_DTYPE
    for kw in (dict(a8=5), dict(a9=-1), dict(a10=0.0)):
        assert b(**kw) == E_ENUM, kw
    for kw in (dict(a5=-1), dict(a6=2000), dict(a7=65)):
        assert b(**kw) == E_SHAPE, kw
    for i in (0, 1, 2, 3, 11):
        assert b(**{f"a{i}": None}) == E_NULL, i
    for i, o in ((0, 2), (1, 2), (2, 2), (3, 4), (11, 8)):
        assert b(**{f"a{i}": FAKE + o}) == E_ALIGN, i
    assert b(a5=0, a0=None) == OK


def test_int4(lib):
    # w, dtype, N, K, group, symmetric, codes, scales, zeros, stream
    q = caller(lib.bsq_quantize_int4, [FAKE, 1, 8, 256, 64, 0, FAKE, FAKE, FAKE, None])
    assert q(a1=7) == E_DTYPE
    assert q(a5=2) == E_ENUM
    for kw in (dict(a2=-1), dict(a2=1 << 31), dict(a3=32), dict(a3=96), dict(a3=32832), dict(a4=16), dict(a4=256)):
        assert q(**kw) == E_SHAPE, kw
    for i in (0, 6, 7, 8):
        assert q(**{f"a{i}": None}) == E_NULL, i
    for kw in (dict(a0=FAKE + 8), dict(a6=FAKE + 4), dict(a7=FAKE + 1)):
        assert q(**kw) == E_ALIGN, kw
    assert q(a2=0, a0=None) == OK
    # codes, scales, zeros, N, K, group, out, out_dtype, stream
    d = caller(lib.bsq_dequantize_int4, [FAKE, FAKE, None, 8, 256, 64, FAKE, 0, None])
    assert d(a7=2) == E_DTYPE
    assert d(a5=48) == E_SHAPE
    for i in (0, 1, 6):
        assert d(**{f"a{i}": None}) == E_NULL, i
    assert d(a6=FAKE + 4) == E_ALIGN
    assert d(a3=0, a0=None) == OK
    # x, dtype, codes, scales, zeros, group, bias, M, N, K, out, out_dtype, ws, bytes, stream
    need = lib.bsq_linear_int4_workspace(500, 300, 256, 64, 1)
    assert need > 0
    c = caller(lib.bsq_linear_int4, [FAKE, 1, FAKE, FAKE, FAKE, 64, None, 500, 300, 256, FAKE, 1, FAKE, need, None])
    assert c(a1=2) == E_DTYPE and c(a11=-1) == E_DTYPE
    for kw in (dict(a5=100), dict(a7=-1), dict(a7=1 << 31), dict(a8=-1), dict(a8=1 << 31), dict(a9=250), dict(a9=0), dict(a9=32832)):
        assert c(**kw) == E_SHAPE, kw
    for i in (0, 2, 3, 10, 12):
        assert c(**{f"a{i}": None}) == E_NULL, i
    for kw in (dict(a0=FAKE + 4), dict(a2=FAKE + 8), dict(a3=FAKE + 1), dict(a6=FAKE + 2), dict(a10=FAKE + 1), dict(a12=FAKE + 8),
               dict(a11=0, a10=FAKE + 2)):
        assert c(**kw) == E_ALIGN, kw
    assert c(a13=need - 1) == E_WORKSPACE
    assert c(a7=0, a0=None) == OK and c(a8=0, a0=None) == OK


def test_int4_workspace(lib):
    w = lib.bsq_linear_int4_workspace
    assert w(1, 4096, 4096, 128, 1) == 0 and w(16, 4096, 4096, 128, 1) == 0
    for bad in ((0, 8, 256, 64, 1), (4, 0, 256, 64, 1), (4, 8, 250, 64, 1), (4, 8, 256, 48, 1), (1 << 31, 8, 256, 64, 1), (-4, 8, 256, 64, 1)):
        assert w(*bad) == 0, bad
    # bounded whatever the sizes
    for M in (1, 17, 64, 65, 200, 5000, (1 << 31) - 1):
        for N in (1, 4099, 100003, (1 << 31) - 1):
            for K, group in ((32, 32), (4096, 128), (32768, 32), (32736, 32)):
                for dtype in (0, 1):
                    assert w(M, N, K, group, dtype) <= 320 << 20, (M, N, K, group, dtype)
    for M, N, K, group, dtype in ((26592, 482364, 32768, 32, 1), (13127, 23388, 32768, 32, 1), (1189, 32112, 9472, 32, 0)):
        assert w(M, N, K, group, dtype) <= 320 << 20  # sizes that K could be split for


def test_logprobs(lib):
    need = lib.bsq_token_logprobs_workspace(4, 1000, 5, 1)
    assert need > 0 and lib.bsq_token_logprobs_workspace(5000, 1000, 0, 1) == 0
    for bad in ((0, 8, 1, 0), (4, 0, 0, 0), (4, (1 << 20) + 1, 0, 0), (4, 100, 65, 0), (4, 100, -1, 0), (-1, 8, 0, 0)):
        assert lib.bsq_token_logprobs_workspace(*bad) == 0, bad
    # logits, dtype, targets, tokens, V, top, logprobs, entropy, stats, top_lp, top_ids, ws, bytes, stream
    c = caller(lib.bsq_token_logprobs, [FAKE, 1, FAKE, 4, 1000, 5, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, need, None])
    assert c(a1=2) == E_DTYPE
    for kw in (dict(a3=-1), dict(a3=1 << 31), dict(a4=0), dict(a4=(1 << 20) + 1), dict(a5=-1), dict(a5=65), dict(a4=4)):
        assert c(**kw) == E_SHAPE, kw
    for i in (0, 2, 6, 7, 8, 9, 10, 11):
        assert c(**{f"a{i}": None}) == E_NULL, i
    for kw in (dict(a0=FAKE + 8), dict(a2=FAKE + 4), dict(a6=FAKE + 2), dict(a7=FAKE + 2), dict(a8=FAKE + 1), dict(a9=FAKE + 2),
               dict(a10=FAKE + 1), dict(a11=FAKE + 8)):
        assert c(**kw) == E_ALIGN, kw
    assert c(a12=need - 1) == E_WORKSPACE
    assert c(a3=0, a0=None) == OK
    # dlogprobs, dentropy, logits, dtype, targets, stats, entropy, tokens, V, dlogits, stream
    b = caller(lib.bsq_token_logprobs_backward, [FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, 4, 100, FAKE, None])
    assert b(a3=2) == E_DTYPE
    assert b(a7=-1) == E_SHAPE and b(a8=0) == E_SHAPE
    for i in (2, 4, 5, 6, 9):
        assert b(**{f"a{i}": None}) == E_NULL, i
    assert b(a0=None, a1=None) == E_NULL
    for i, o in ((0, 2), (1, 2), (2, 8), (4, 4), (5, 2), (6, 2), (9, 8)):
        assert b(**{f"a{i}": FAKE + o}) == E_ALIGN, i
    assert b(a7=0, a0=None, a2=None) == OK
