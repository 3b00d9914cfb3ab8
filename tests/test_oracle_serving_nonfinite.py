"""The 8-bit quantizer's oracle for rows without finite codes (no GPU)."""
import numpy as np

from oracle import serving as S


def test_quantize_int8_rows_without_codes():
    x = np.array([[1.0, np.nan], [np.inf, 1.0], [-np.inf, np.nan], [3e38, 1.0]], dtype=np.float32)
    q, s = S.quantize_int8(x)
    assert np.isnan(s[:3]).all() and np.isfinite(s[3]) and q[3].tolist() == [127, 0]
