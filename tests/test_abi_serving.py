"""Argument checks of the router, few-token expert layer and 8-bit product entry
points, on the host before any HIP call (no GPU needed)."""
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


def test_gate(lib):
    # logits, dtype, tokens, E, k, renorm, weights, ids, stream
    c = caller(lib.bsq_moe_gate, [FAKE, 0, 4, 64, 8, 1, FAKE, FAKE, None])
    assert c(a1=2) == E_DTYPE
    assert c(a5=2) == E_ENUM
    for kw in (dict(a2=-1), dict(a3=0), dict(a3=1025), dict(a4=0), dict(a4=65), dict(a3=7), dict(a2=1 << 31)):
        assert c(**kw) == E_SHAPE, kw
    for kw in (dict(a0=None), dict(a6=None), dict(a7=None)):
        assert c(**kw) == E_NULL, kw
    for kw in (dict(a0=FAKE + 8), dict(a6=FAKE + 2), dict(a7=FAKE + 1)):
        assert c(**kw) == E_ALIGN, kw
    assert c(a2=0, a0=None, a6=None, a7=None) == OK
    # dweights, weights, ids, logits, dtype, tokens, E, k, renorm, dlogits, stream
    b = caller(lib.bsq_moe_gate_backward, [FAKE, FAKE, FAKE, FAKE, 1, 4, 64, 8, 0, FAKE, None])
    assert b(a4=9) == E_DTYPE
    assert b(a8=-1) == E_ENUM
    assert b(a7=65) == E_SHAPE
    for i in (0, 1, 2, 3, 9):
        assert b(**{f"a{i}": None}) == E_NULL, i
    for i in (3, 9):
        assert b(**{f"a{i}": FAKE + 4}) == E_ALIGN, i
    for i in (0, 1, 2):
        assert b(**{f"a{i}": FAKE + 2}) == E_ALIGN, i
    assert b(a5=0, a0=None) == OK


def test_moe_few(lib):
    # x, dtype, T, H, F, E, k, ids, weights, 13 codes, scales, outer, 2 codes, scales, outer, out, ws, bytes, stream
    need = lib.bsq_moe_few_nvfp4_workspace(4, 256, 128, 8, 2)
    assert need > 0
    c = caller(lib.bsq_moe_few_nvfp4, [FAKE, 1, 4, 256, 128, 8, 2] + [FAKE] * 10 + [need, None])
    assert c(a1=5) == E_DTYPE
    limit = _lib.MOE_FEW_MAX_PAIRS
    for kw in (dict(a2=-1), dict(a2=limit // 2 + 1), dict(a3=264), dict(a3=0), dict(a3=32784), dict(a4=8), dict(a4=0),
               dict(a4=32784), dict(a5=0), dict(a5=1025), dict(a6=0), dict(a6=65)):
        assert c(**kw) == E_SHAPE, kw
    for i in range(7, 17):
        assert c(**{f"a{i}": None}) == E_NULL, i
    assert c(a0=None) == E_NULL
    for i in (0, 9, 10, 12, 13, 15, 16):
        assert c(**{f"a{i}": FAKE + 8}) == E_ALIGN, i
    for i in (7, 8, 11, 14):
        assert c(**{f"a{i}": FAKE + 2}) == E_ALIGN, i
    assert c(a17=need - 1) == E_WORKSPACE
    assert c(a2=0, a0=None) == OK
    assert lib.bsq_moe_few_nvfp4_workspace(limit + 1, 256, 128, 8, 1) == 0
    assert lib.bsq_moe_few_nvfp4_workspace(1 << 62, 256, 128, 8, 1 << 62) == 0


def test_int8(lib):
    # x, dtype, rows, cols, codes, scales, stream
    for fn in (lib.bsq_quantize_int8, lib.bsq_swiglu_quantize_int8):
        q = caller(fn, [FAKE, 1, 4, 32, FAKE, FAKE, None])
        assert q(a1=2) == E_DTYPE
        for kw in (dict(a2=-1), dict(a2=1 << 31), dict(a3=0), dict(a3=24), dict(a3=32784)):
            assert q(**kw) == E_SHAPE, kw
        for i in (0, 4, 5):
            assert q(**{f"a{i}": None}) == E_NULL
        for i in (0, 4):
            assert q(**{f"a{i}": FAKE + 8}) == E_ALIGN
        assert q(a5=FAKE + 2) == E_ALIGN
        assert q(a2=0, a0=None) == OK
    # a, sa, b, sb, bias, M, N, K, out, dtype, stream
    g = caller(lib.bsq_gemm_int8, [FAKE, FAKE, FAKE, FAKE, None, 4, 8, 32, FAKE, 1, None])
    assert g(a9=3) == E_DTYPE
    for kw in (dict(a5=-1), dict(a6=-1), dict(a7=0), dict(a7=24), dict(a7=131072), dict(a5=1 << 31), dict(a6=1 << 31),
               dict(a5=(1 << 31) - 1, a6=(1 << 31) - 1)):
        assert g(**kw) == E_SHAPE, kw
    for i in (0, 1, 2, 3, 8):
        assert g(**{f"a{i}": None}) == E_NULL
    for i in (0, 2):
        assert g(**{f"a{i}": FAKE + 8}) == E_ALIGN
    for i in (1, 3, 4):
        assert g(**{f"a{i}": FAKE + 2}) == E_ALIGN
    assert g(a8=FAKE + 1) == E_ALIGN
    assert g(a8=FAKE + 2, a9=0) == E_ALIGN
    assert g(a5=0, a0=None) == OK
    assert g(a6=0, a2=None) == OK
    # x, dtype, b, sb, bias, M, N, K, out, out_dtype, ws, bytes, stream
    need = lib.bsq_linear_int8_workspace(20, 32)
    assert need > 0 and lib.bsq_linear_int8_workspace(1, 4096) == 0
    l = caller(lib.bsq_linear_int8, [FAKE, 1, FAKE, FAKE, None, 20, 8, 32, FAKE, 1, FAKE, need, None])
    assert l(a1=2) == E_DTYPE
    assert l(a9=2) == E_DTYPE
    assert l(a7=32784) == E_SHAPE
    for i in (0, 2, 3, 8, 10):
        assert l(**{f"a{i}": None}) == E_NULL
    for i in (0, 2, 10):
        assert l(**{f"a{i}": FAKE + 8}) == E_ALIGN
    assert l(a11=need - 1) == E_WORKSPACE
    assert l(a5=0, a0=None) == OK


def test_workspace_queries_of_impossible_sizes(lib):
    assert lib.bsq_linear_int8_workspace(-1, 32) == 0
    assert lib.bsq_linear_int8_workspace(16, 1 << 40) >= 16 << 40
    assert lib.bsq_moe_few_nvfp4_workspace(4, 32768, 32768, 8, 2) > lib.bsq_moe_few_nvfp4_workspace(4, 4096, 4096, 8, 2)
    assert lib.bsq_moe_few_nvfp4_workspace(4, 32784, 64, 8, 2) == 0
