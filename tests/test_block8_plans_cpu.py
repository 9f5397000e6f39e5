"""The products that test_block8_forms_gpu.py runs take the paths they are
there for: asked of the library's own rule, which needs no GPU."""
import ctypes

import pytest

import int8_quantized_matmul_outlier_b200 as m
from tests._block8_plans import PIPELINES

SMS = 148


def pair_width(M, K, N):
    f = m.lib()._ZN4i8mm16block_pair_widthEllli  # i8mm::block_pair_width(M, N, K, num_sms)
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int64] * 3 + [ctypes.c_int]
    return f(M, N, K, SMS)


@pytest.mark.parametrize("M,K,N,width,groups,rounds", PIPELINES)
def test_tile_width_and_rounds(M, K, N, width, groups, rounds):
    assert pair_width(M, K, N) == width
    tiles = -(-M // 256) * -(-N // width)
    assert -(-tiles // (SMS // 2)) == rounds and -(-K // 128) == groups


def test_the_paths_that_matter_are_among_them():
    """For each width: an odd and an even number of groups over several boxes
    of 16, which swap the producers' and the scale buffers' turns from tile to
    tile or keep them; more than two boxes; ragged edges."""
    for width in (128, 256):
        of = [p for p in PIPELINES if p[3] == width]
        assert all(p[4] > 16 and p[5] > 1 for p in of)
        assert {p[4] % 2 for p in of} == {0, 1} and {-(-p[4] // 16) % 2 for p in of} == {0, 1}
        assert any(p[0] % 256 and p[1] % 128 and p[2] % width for p in of)
