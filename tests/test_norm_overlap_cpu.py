"""The norms refuse an h that lies shifted over its own row of x or of the residual, on
the host: elements of the row are read while others of its h are stored.  (Only
refusals: the addresses are no memory.)"""
import ctypes

import pytest

from w8a8_int8_quantized_i8_gb300 import binding

FAR = 1 << 28
X, RES, CODES, SCALES, ROWS, H = ((i + 1) * FAR for i in range(6))
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def _four_bits(lib, M, K, ldx, ldr, h, ldh):
    return lib.i8_add_rmsnorm_quant_fp4(P(X), M, K, ldx, P(RES), ldr, None, 1e-6, 0, P(CODES), P(SCALES), P(ROWS), P(h),
                                        ldh, None)


def _eight_bits(lib, M, K, ldx, ldr, h, ldh):
    return lib.i8_add_rmsnorm_quant_act_pertoken(P(X), M, K, ldx, P(RES), ldr, None, 1e-6, 0, P(CODES), K, P(ROWS), P(h), ldh,
                                                 None)


@pytest.mark.parametrize("call", [_four_bits, _eight_bits])
@pytest.mark.parametrize("base", [X, RES])
@pytest.mark.parametrize("K", [64, 32768])
@pytest.mark.parametrize("M", [1, 2, 5])
def test_h_shifted_inside_its_row(lib, call, base, K, M):
    wide = 4 * K
    for shift in (16, 2 * K - 16, -16, 16 - 2 * K):
        assert call(lib, M, K, wide, wide, base + shift, wide) == 1, shift


@pytest.mark.parametrize("call", [_four_bits, _eight_bits])
@pytest.mark.parametrize("base", [X, RES])
def test_a_later_row_shifted_by_another_stride(lib, call, base):
    """Rows of h that begin in the gaps and come to lie over x's own rows."""
    K, ldx = 64, 512
    for ldh in (ldx - 8, ldx + 8):
        for first in range(2 * K, 2 * ldx - 2 * K + 1, 64):
            h = base - first if ldh > ldx else base + first     # (bytes; drifts over its row by 16 a row)
            rows = first // 16 + 2
            assert call(lib, rows, K, ldx, ldx, h, ldh) == 1, (ldh, first)
    # in the gaps throughout, and in place: nothing to refuse (no rows: nothing is queued)
    assert call(lib, 0, K, ldx, ldx, base + 16, ldx) == 0


def test_a_longer_row_than_the_eight_bit_norm_takes(lib):
    K = 65536
    for base in (X, RES):
        assert _four_bits(lib, 1, K, K, K, base + 16, K) == 1 and _four_bits(lib, 3, K, 2 * K, 2 * K, base - 32, 2 * K) == 1
