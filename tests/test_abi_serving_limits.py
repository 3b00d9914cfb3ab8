"""Largest sizes that the serving entry points take, on the host (no GPU needed)."""
import os

import pytest

from block_scaled_bit_quantize_amd import _lib

E_SHAPE = 2
FAKE = 0x10000  # never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.library_path()):
        from block_scaled_bit_quantize_amd.build import build
        build()
    return _lib.load_library()


def test_channels_of_the_int8_products(lib):
    for n in ((1 << 31) - 255, (1 << 31) - 1):  # a launch would not take 128 rows of them
        assert lib.bsq_gemm_int8(FAKE, FAKE, FAKE, FAKE, None, 4, n, 32, FAKE, 1, None) == E_SHAPE
        assert lib.bsq_linear_int8(FAKE, 1, FAKE, FAKE, None, 1, n, 32, FAKE, 1, None, 0, None) == E_SHAPE
