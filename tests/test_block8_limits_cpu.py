"""The ends of the documented ranges of the e4m3 entry points, on the host."""
import ctypes

import pytest

import int8_quantized_matmul_outlier_b200 as m

P = ctypes.c_void_p(1 << 20)  # never dereferenced: the output lies on the input and the call is refused
S = ctypes.c_void_p(1 << 45)


@pytest.mark.parametrize("lds", [1 << 31, (1 << 31) + 4, 1 << 32])
@pytest.mark.parametrize("M", [(1 << 31) - 1, (1 << 31) - 3, 5])
def test_the_scales_of_the_most_rows_have_a_stride(M, lds):
    L = m.lib()
    assert L.int8mm_block_quantize(P, 0, M, 16, 16, P, S, lds, None) == m.INT8MM_ERR_INVALID_ARG
    assert m.int8mm_last_error() == "codes overlaps X"
    assert L.int8mm_block_rms_norm(P, 16, None, 0, S, 0, M, 16, 1e-6, None, None, P, S, lds, None) == \
        m.INT8MM_ERR_INVALID_ARG
    assert m.int8mm_last_error() == "codes overlaps X"


@pytest.mark.parametrize("M,lds", [((1 << 31) - 1, (1 << 31) - 4), (5, (1 << 32) + 4), (5, (1 << 31) + 2)])
def test_other_strides_of_the_scales_are_refused(M, lds):
    assert m.lib().int8mm_block_quantize(P, 0, M, 16, 16, P, S, lds, None) == m.INT8MM_ERR_INVALID_ARG
    assert "scales: stride" in m.int8mm_last_error()
