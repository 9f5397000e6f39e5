"""Failure detection of the e4m3 products without a fault: a test-only switch
leaves out one kind of arrival (nothing else changes), the waits for it run out
after the handle's limit, the kernel drains and exits, the status reads TIMEOUT
once, and the next product has the right bits."""
import pytest
import torch

import int8_quantized_matmul_outlier_b200 as m
from tests.test_block8_gpu import F16, problem

pytestmark = pytest.mark.gpu

WAITS = [
    # (what is left out, M, K, N)
    ("scales", 1, 8192, 16384),    # few rows, one box after another or one tile after another
    ("scales", 40, 8192, 16384),
    ("meeting", 9, 20480, 144),    # few columns: K split over clusters of 8
    ("meeting", 64, 12288, 272),
    ("scales", 700, 2176, 8192),   # CTA pairs, 128-wide tiles
    ("scales", 1024, 2176, 8192),  # 256-wide tiles
]


@pytest.mark.parametrize("what,M,K,N", WAITS)
def test_a_product_wait_that_runs_out_is_reported_and_the_handle_recovers(what, M, K, N):
    bits = {"scales": m.INT8MM_BLOCK_TEST_SKIP_SCALES, "meeting": m.INT8MM_BLOCK_TEST_SKIP_MEETING}[what]
    _, w, codes, scales = problem(M, K, N, F16, M)
    _, other, c2, s2 = problem(M, 272, 144, F16, M + 1)
    want, want2 = m.int8mm_block_matmul(w, codes, scales), m.int8mm_block_matmul(other, c2, s2)
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK
    with pytest.raises(m.Int8mmError):
        m.int8mm_block_set_test_skip(w, 4)  # not a known arrival
    m.int8mm_block_set_wait_limit(w, 1_000_000)
    m.int8mm_block_set_test_skip(w, bits)
    m.int8mm_block_matmul(w, codes, scales)
    y2 = m.int8mm_block_matmul(other, c2, s2)  # behind it on the stream
    assert m.int8mm_block_get_status(w) == m.INT8MM_ERR_TIMEOUT
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK  # reading the word cleared it
    assert m.int8mm_block_get_status(other) == m.INT8MM_OK and torch.equal(y2, want2)
    m.int8mm_block_set_test_skip(w, 0)
    m.int8mm_block_set_wait_limit(w, 2_000_000_000)
    for _ in range(3):
        assert torch.equal(m.int8mm_block_matmul(w, codes, scales), want)
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK
