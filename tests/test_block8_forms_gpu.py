"""Forms of the e4m3 operators that need sizes of their own to be reached, on
the GPU against the plain forms (tests/_block8.py)."""
import pytest
import torch

import int8_quantized_matmul_outlier_b200 as m
from tests import _block8 as ref
from tests._block8_plans import PIPELINES
from tests.test_block8_gpu import BF16, F16, acts, bits, dev, gen, problem, same_quantised

pytestmark = pytest.mark.gpu


def test_the_most_rows():
    """2^31 - 1 rows of 16 columns: the first rows, some in the middle and the
    last ones."""
    M, K, N = 2 ** 31 - 1, 16, 16
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 125 << 30:
        pytest.skip("needs 125 GB of device memory")
    parts = (slice(0, 300), slice(2 ** 30 - 150, 2 ** 30 + 150), slice(M - 600, M))
    x = torch.empty(M, K, dtype=BF16, device=dev()).normal_(generator=gen(1))
    codes, scales = m.int8mm_block_quantize(x)
    for p in parts:
        same_quantised(codes[p], scales[p], *ref.quantise(x[p]))
    wt = (1 + 0.3 * torch.randn(K, generator=gen(2), device="cuda")).to(BF16)
    del codes, scales
    codes, scales, _, _ = m.int8mm_block_rms_norm(x, wt)
    for p in parts:
        c, s, _, _ = m.int8mm_block_rms_norm(x[p].clone(), wt)
        assert torch.equal(bits(codes[p]), bits(c)) and torch.equal(scales[p], s)
    del x
    torch.cuda.empty_cache()
    w = m.int8mm_block_prepare_weight((torch.randn(K, N, generator=gen(3), device="cuda") * 0.02).to(BF16))
    y = m.int8mm_block_matmul(w, codes, scales, dtype=BF16)
    wc, ws = m.int8mm_block_weight_codes(w)
    for p in parts:
        ref.check_product(y[p], codes[p], scales[p], wc, ws, None, K)
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK
    del y, codes, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("sx,sr", [((2, 3), (6,)), ((6,), (2, 3)), ((2, 3), (1, 2, 3)), ((1, 6), (6,)), ((), (1,))])
def test_norm_layer_takes_rows_for_a_batch(sx, sr):
    """x and the residual of one row order, one of them flattened."""
    norm = m.RMSNormBlock8bit(272)
    n = max(torch.Size(sx).numel(), 1)
    x, r = (torch.randn(n, 272, generator=gen(i), device="cuda").half() for i in (1, 2))
    want = m.int8mm_block_rms_norm(x, norm.weight.data, norm.eps, residual=r)
    (codes, scales), out = norm(x.view(*sx, 272), r.view(*sr, 272))
    assert out.shape == (*sx, 272) and torch.equal(out.view(n, 272), want[2])
    assert torch.equal(bits(codes), bits(want[0])) and torch.equal(scales, want[1])


# ------------------------------------------------------- every form of the kernels
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("M,K", [(2100, 1024), (1400, 2064), (2000, 1552), (600, 5136), (300, 12288)])
def test_quantise_runs_of_several_vectors(M, K, dtype, wide):
    """2 and 4 vectors per lane, with a full and a ragged last run."""
    x = acts(M, K, dtype, M + K, wide)
    codes, scales = m.int8mm_block_quantize(x)
    same_quantised(codes, scales, *ref.quantise(x))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("M,K", [
    (300, 272), (297, 512), (299, 528), (300, 1024),                          # a warp per row
    (300, 1040), (300, 2064), (300, 4112), (300, 6160), (300, 8192), (300, 9216), (300, 12288), (300, 13328),
    (300, 16384),                                                             # 256 threads, 1 to 8 vectors each
    (300, 16400), (300, 32784),                                               # many rows past those
    (1, 2064), (9, 4096), (1, 4112), (9, 8192), (295, 8176), (9, 16384), (9, 32768)])  # few rows
def test_norm_threads_and_vectors(M, K, dtype, with_residual):
    x = acts(M, K, dtype, M + K)
    r = acts(M, K, dtype, M + K + 1) if with_residual else None
    wt = (1 + 0.3 * torch.randn(K, generator=gen(K), device="cuda")).to(dtype)
    codes, scales, ro, y = m.int8mm_block_rms_norm(x, wt, 1e-5, residual=r, normed=True)
    h, y64 = ref.norm(x, r, wt, 1e-5)
    assert ro is None if r is None else torch.equal(ro, h)
    ref.check_normed(y, y64)
    ref.check_quantised(codes, scales, y64)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,N", [p[:3] for p in PIPELINES])
def test_product_over_several_tiles_and_boxes_of_scales(M, K, N, dtype):
    x, w, codes, scales = problem(M, K, N, dtype, M + K + N)
    bias = (torch.randn(N, generator=gen(7), device="cuda") * 0.5).to(dtype)
    y = m.int8mm_block_matmul(w, codes, scales, bias=bias, dtype=dtype)
    ref.check_product(y, codes, scales, *m.int8mm_block_weight_codes(w), bias, K)
    for _ in range(5):
        assert torch.equal(m.int8mm_block_matmul(w, codes, scales, bias=bias, dtype=dtype), y)
    assert torch.equal(m.int8mm_block_forward(w, x, bias=bias), y)
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK


@pytest.mark.parametrize("K", [256, 1040, 12288])
def test_norm_where_the_squares_leave_fp32(K):
    """As the header says: 0 past the range, Inf (NaN for 0) below it without an eps; other rows are not touched."""
    x = acts(6, K, BF16, 1)
    want = m.int8mm_block_rms_norm(x, torch.ones(K, dtype=BF16, device=dev()), 0.0, normed=True)
    x[1], x[3], x[4] = 2.0 ** 70, 2.0 ** -80, 0.0
    codes, scales, _, y = m.int8mm_block_rms_norm(x, torch.ones(K, dtype=BF16, device=dev()), 0.0, normed=True)
    assert (y[1] == 0).all() and (codes[1].float() == 0).all() and (scales[1] == 0).all()
    assert (y[3] == float("inf")).all() and y[4].isnan().all() and scales[4].isnan().all()
    keep = [0, 2, 5]
    assert torch.equal(y[keep], want[3][keep]) and torch.equal(scales[keep], want[1][keep])
    assert torch.equal(bits(codes[keep]), bits(want[0][keep]))
