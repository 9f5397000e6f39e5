"""The e4m3 block-scaled entry points on the host: bad arguments are refused
before anything is enqueued, in C and in Python."""
import ctypes

import pytest
import torch

import int8_quantized_matmul_outlier_b200 as m
from int8_quantized_matmul_outlier_b200 import block

P = 1 << 20  # 16-byte aligned, never dereferenced: the checks come first
BIG = 1 << 28  # distance between fake buffers


def buf(i, off=0):
    return ctypes.c_void_p(P + i * BIG + off)


BAD_PREPARE = [
    (buf(0), 2, 128, 128, m.INT8MM_ERR_INVALID_ARG),                   # no such type
    (None, 0, 128, 128, m.INT8MM_ERR_INVALID_ARG),
    (buf(0), 0, 120, 128, m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (buf(0), 0, 0, 128, m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (buf(0), 0, m.MAX_K + 16, 128, m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (buf(0), 0, 128, 8, m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (buf(0), 0, 128, 24, m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (buf(0), 0, 128, (1 << 31) - 16, m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (buf(0), 0, 65536, 1 << 22, m.INT8MM_ERR_UNSUPPORTED_SHAPE),       # more rows than the layout can index
    (buf(0, 8), 0, 128, 128, m.INT8MM_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("W,dtype,K,N,status", BAD_PREPARE)
def test_prepare_refuses(W, dtype, K, N, status):
    L = m.lib()
    out = ctypes.c_void_p(1234)
    assert L.int8mm_block_prepare_weight(W, dtype, K, N, None, ctypes.byref(out)) == status
    assert out.value is None and m.int8mm_last_error()
    if dtype == 0:
        out = ctypes.c_void_p(1234)
        assert L.int8mm_block_prepare_codes(W, buf(1), K, N, None, ctypes.byref(out)) == status
        assert out.value is None


def test_prepare_refuses_missing_outputs_and_scales():
    L = m.lib()
    out = ctypes.c_void_p(1234)
    assert L.int8mm_block_prepare_weight(buf(0), 0, 128, 128, None, None) == m.INT8MM_ERR_INVALID_ARG
    assert L.int8mm_block_prepare_codes(buf(0), None, 128, 128, None, ctypes.byref(out)) == m.INT8MM_ERR_INVALID_ARG
    assert out.value is None


def quantise_args(**kw):
    a = dict(X=buf(0), dtype=0, M=5, K=256, ldx=256, codes=buf(1), scales=buf(2), lds=8)
    a.update(kw)
    return [*a.values(), None]


BAD_QUANTISE = [
    (dict(dtype=-1), m.INT8MM_ERR_INVALID_ARG),
    (dict(M=-1), m.INT8MM_ERR_INVALID_ARG),
    (dict(M=1 << 31), m.INT8MM_ERR_INVALID_ARG),
    (dict(K=8), m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (dict(K=136, ldx=136), m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (dict(X=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(codes=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(scales=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(ldx=248), m.INT8MM_ERR_INVALID_ARG),
    (dict(ldx=260), m.INT8MM_ERR_ALIGNMENT),
    (dict(X=buf(0, 2)), m.INT8MM_ERR_ALIGNMENT),
    (dict(codes=buf(1, 4)), m.INT8MM_ERR_ALIGNMENT),
    (dict(scales=buf(2, 4)), m.INT8MM_ERR_ALIGNMENT),
    (dict(lds=4), m.INT8MM_ERR_INVALID_ARG),
    (dict(lds=6), m.INT8MM_ERR_INVALID_ARG),
    (dict(codes=buf(0, 512)), m.INT8MM_ERR_INVALID_ARG),    # overlaps X
    (dict(scales=buf(1, 1264)), m.INT8MM_ERR_INVALID_ARG),  # overlaps the end of codes (5 x 256 bytes)
]


@pytest.mark.parametrize("change,status", BAD_QUANTISE)
def test_quantise_refuses(change, status):
    assert m.lib().int8mm_block_quantize(*quantise_args(**change)) == status
    assert m.int8mm_last_error()


def norm_args(**kw):
    a = dict(X=buf(0), ldx=256, residual=buf(1), ldr=256, weight=buf(2), dtype=0, M=5, K=256, eps=1e-6,
             residual_out=buf(3), normed=buf(4), codes=buf(5), scales=buf(6), lds=8)
    a.update(kw)
    return [*a.values(), None]


BAD_NORM = [
    (dict(dtype=7), m.INT8MM_ERR_INVALID_ARG),
    (dict(M=-3), m.INT8MM_ERR_INVALID_ARG),
    (dict(K=m.MAX_K + 16), m.INT8MM_ERR_UNSUPPORTED_SHAPE),
    (dict(eps=-1.0), m.INT8MM_ERR_INVALID_ARG),
    (dict(eps=float("nan")), m.INT8MM_ERR_INVALID_ARG),
    (dict(eps=float("inf")), m.INT8MM_ERR_INVALID_ARG),
    (dict(residual=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(residual_out=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(codes=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(scales=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(codes=None, scales=None, normed=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(weight=None), m.INT8MM_ERR_INVALID_ARG),
    (dict(weight=buf(2, 2)), m.INT8MM_ERR_ALIGNMENT),
    (dict(ldr=260), m.INT8MM_ERR_ALIGNMENT),
    (dict(normed=buf(4, 8)), m.INT8MM_ERR_ALIGNMENT),
    (dict(lds=2), m.INT8MM_ERR_INVALID_ARG),
    (dict(normed=buf(0)), m.INT8MM_ERR_INVALID_ARG),                    # onto X
    (dict(residual_out=buf(1, 16)), m.INT8MM_ERR_INVALID_ARG),          # shifted against residual
    (dict(residual_out=buf(0), ldx=264), m.INT8MM_ERR_INVALID_ARG),     # in place on strided rows
    (dict(residual_out=buf(4)), m.INT8MM_ERR_INVALID_ARG),              # onto normed
    (dict(codes=buf(2)), m.INT8MM_ERR_INVALID_ARG),                     # onto the weight
]


@pytest.mark.parametrize("change,status", BAD_NORM)
def test_norm_refuses(change, status):
    assert m.lib().int8mm_block_rms_norm(*norm_args(**change)) == status
    assert m.int8mm_last_error()


def test_empty_inputs_are_no_ops():
    L = m.lib()
    assert L.int8mm_block_quantize(*quantise_args(M=0, X=None, codes=None, scales=None)) == m.INT8MM_OK
    assert L.int8mm_block_rms_norm(*norm_args(M=0)) == m.INT8MM_OK


def test_calls_on_an_unknown_handle_are_refused():
    L = m.lib()
    bogus = ctypes.c_void_p(0xdead0)
    assert L.int8mm_block_matmul(bogus, buf(0), buf(1), 8, 5, None, buf(2), 0, None) == m.INT8MM_ERR_INVALID_ARG
    assert "handle" in m.int8mm_last_error()
    assert L.int8mm_block_weight_codes(bogus, None, None, None) == m.INT8MM_ERR_INVALID_ARG
    assert L.int8mm_block_forward(bogus, buf(0), 128, 5, None, buf(1), 0, buf(2), 1 << 20, None) == \
        m.INT8MM_ERR_INVALID_ARG
    assert L.int8mm_block_forward_scratch(bogus, 5, ctypes.byref(ctypes.c_size_t())) == m.INT8MM_ERR_INVALID_ARG
    assert L.int8mm_block_get_status(bogus) == m.INT8MM_ERR_INVALID_ARG
    assert L.int8mm_block_set_wait_limit(bogus, 10 ** 9) == m.INT8MM_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert L.int8mm_block_weight_bytes(bogus, ctypes.byref(n)) == m.INT8MM_ERR_INVALID_ARG
    L.int8mm_block_free(None)   # no-op
    L.int8mm_block_free(bogus)  # unknown handle: no-op


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        m.int8mm_block_quantize(x)
    with pytest.raises(ValueError):
        m.int8mm_block_rms_norm(x, torch.ones(128, dtype=torch.float16))
    with pytest.raises(ValueError):
        m.int8mm_block_prepare_weight(x)
    with pytest.raises(ValueError):
        m.int8mm_block_prepare_codes(x.to(torch.float8_e4m3fn), torch.ones(1, 1))


@pytest.mark.parametrize("M,K", [(1, 128), (1, 400), (5, 128), (5, 1040), (8, 256), (513, 20480)])
def test_the_scales_layout_is_accepted_as_made(M, K):
    G = block._groups(K)
    s = block._new_scales(M, G, torch.device("cpu"))
    assert tuple(s.shape) == (M, G)
    lds = block._scales_ld(s, M, G, torch.device("cpu"))
    assert lds >= M and lds % 4 == 0 and lds == (M + 3) // 4 * 4
    wide = torch.zeros(G, 4 * M + 4).t()[:M]  # a longer distance between groups
    assert block._scales_ld(wide, M, G, torch.device("cpu")) == 4 * M + 4


def test_other_scales_layouts_are_refused():
    cpu = torch.device("cpu")
    for s in (torch.zeros(5, 3),                      # row-major
              torch.zeros(3, 5).t(),                  # groups 5 apart
              torch.zeros(3, 8, dtype=torch.float64).t()[:5],
              torch.zeros(3, 8).t()[:4],              # another M
              torch.zeros(2, 8).t()[:5]):             # another G
        with pytest.raises(ValueError):
            block._scales_ld(s, 5, 3, cpu)
