"""Forms of the e4m3 operators that need sizes of their own to be reached, on
the GPU against the plain forms (tests/_block8.py)."""
import pytest
import torch

import int8_quantized_matmul_outlier_b200 as m
from tests import _block8 as ref
from tests.test_block8_gpu import BF16, F16, bits, dev, gen, same_quantised

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
