"""The e4m3 block-scaled operators on the GPU against plain forms: the
quantisers bit for bit, norms and products against 64 bits within tolerances
that count roundings (tests/_block8.py)."""
import ctypes
import threading

import pytest
import torch

import int8_quantized_matmul_outlier_b200 as m
from tests import _block8 as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def dev():
    return torch.device("cuda", torch.cuda.current_device())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def acts(M, K, dtype, seed, wide=False):
    """Normal values with a few large columns; `wide`: exponents all over the type's range, zeros among them."""
    g = gen(seed)
    x = torch.randn(M, K, generator=g, device="cuda")
    if wide:
        e = torch.randint(-20 if dtype == F16 else -120, 14, (M, K), generator=g, device="cuda")
        x = torch.where(torch.rand(M, K, generator=g, device="cuda") < 0.1, 0.0, torch.ldexp(x.clamp(-1.9, 1.9), e))
    else:
        x[:, torch.randperm(K, generator=g, device="cuda")[:3]] *= 60
    return x.to(dtype)


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int32)


def same_quantised(codes, scales, c_ref, s_ref):
    """Bit for bit; a NaN may be any NaN."""
    codes, scales = codes.cpu(), scales.cpu().contiguous()
    cn, sn = c_ref.float().isnan(), s_ref.isnan()
    assert torch.equal(codes.float().isnan(), cn) and torch.equal(scales.isnan(), sn)
    assert torch.equal(bits(codes.contiguous())[~cn], bits(c_ref.contiguous())[~cn])
    assert torch.equal(scales[~sn], s_ref.contiguous()[~sn])


# ------------------------------------------------------------------ quantise
Q_SHAPES = [(1, 16), (1, 128), (1, 12288), (3, 144), (5, 1040), (7, 65536), (64, 256), (129, 784), (300, 5120),
            (1000, 2064), (20000, 48)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("M,K", Q_SHAPES)
def test_quantise(M, K, dtype, wide):
    x = acts(M, K, dtype, M + K, wide)
    codes, scales = m.int8mm_block_quantize(x)
    assert codes.shape == (M, K) and scales.shape == (M, ref.groups(K))
    same_quantised(codes, scales, *ref.quantise(x))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_quantise_values_where_it_can_go_wrong(dtype):
    """Zero groups, a single value, the largest and smallest numbers, ties."""
    fi = torch.finfo(dtype)
    x = torch.zeros(12, 400, dtype=torch.float64)
    x[1, 3] = 1.0
    x[2, 5] = -fi.max
    x[2, 6] = fi.max
    x[3, 300] = 2.0 ** (-24 if dtype == F16 else -133)  # the smallest subnormal
    x[4, :128] = torch.arange(128) * 2.0 ** -6 - 1     # many ties of e4m3 once scaled
    x[4, 0] = 448.0
    x[5, :] = 448.0 * torch.arange(400) / 400
    x[6, 399] = 3.0                                     # the short last group
    x[7, :] = 2.0 ** -14
    x[8, 128:256] = torch.linspace(-240, 448, 128)
    x[9, 0] = 1e-30 if dtype == BF16 else 1e-7
    x[10, 0] = 2.0 ** -101 if dtype == BF16 else 1e-6   # below the floor of a group's maximum
    x[11] = torch.randn(400, generator=torch.Generator().manual_seed(1)) * 1e-5
    x = x.to(dtype).cuda()
    codes, scales = m.int8mm_block_quantize(x)
    same_quantised(codes, scales, *ref.quantise(x))
    assert (scales[0] == 0).all() and (codes[0].float() == 0).all()


def test_quantise_nan_and_inf_stay_in_their_group():
    x = acts(6, 384, BF16, 3)
    x[1, 130], x[2, 0], x[3, 383], x[4, 200] = float("nan"), float("inf"), float("-inf"), float("nan")
    x[4, 201] = float("inf")
    codes, scales = m.int8mm_block_quantize(x)
    c, s = ref.quantise(x)
    same_quantised(codes, scales, c, s)
    bad = torch.zeros(6, 3, dtype=torch.bool)
    bad[1, 1] = bad[2, 0] = bad[3, 2] = bad[4, 1] = True
    assert torch.equal(~scales.cpu().isfinite(), bad)


@pytest.mark.parametrize("ld", [272, 1024])
def test_quantise_strided_rows(ld):
    x = acts(33, ld, F16, 5)[:, 8:264]
    codes, scales = m.int8mm_block_quantize(x)
    same_quantised(codes, scales, *ref.quantise(x))
    one = x[4:5]
    same_quantised(*m.int8mm_block_quantize(one), *ref.quantise(one))


def test_refusals_of_gpu_arguments():
    x = acts(8, 256, F16, 1)
    w = m.int8mm_block_prepare_weight(acts(256, 64, F16, 2))
    codes, scales = m.int8mm_block_quantize(x)
    with pytest.raises(ValueError):
        m.int8mm_block_quantize(x.float())
    with pytest.raises(ValueError):
        m.int8mm_block_quantize(x.t())
    with pytest.raises(m.Int8mmError):
        m.int8mm_block_quantize(acts(8, 264, F16, 1)[:, 1:257])   # rows not 16-byte aligned
    with pytest.raises(m.Int8mmError):
        m.int8mm_block_quantize(acts(8, 200, F16, 1))             # K not a multiple of 16
    with pytest.raises(ValueError):
        m.int8mm_block_rms_norm(x, torch.ones(256, dtype=BF16, device=dev()))
    with pytest.raises(ValueError):
        m.int8mm_block_rms_norm(x, torch.ones(256, dtype=F16, device=dev()), residual=x[:4])
    with pytest.raises(ValueError):
        m.int8mm_block_rms_norm(x, torch.ones(256, dtype=F16, device=dev()), codes=False)
    with pytest.raises(ValueError):
        m.int8mm_block_matmul(w, codes, scales.contiguous())      # row-major scales
    with pytest.raises(ValueError):
        m.int8mm_block_matmul(w, codes[:4], scales)
    with pytest.raises(ValueError):
        m.int8mm_block_matmul(w, codes, scales, dtype=torch.float32)
    with pytest.raises(ValueError):
        m.int8mm_block_matmul(w, codes, scales, bias=torch.zeros(64, dtype=BF16, device=dev()))
    with pytest.raises(ValueError):
        m.int8mm_block_matmul(w, codes, scales, Y=torch.empty(8, 128, dtype=F16, device=dev())[:, :64])
    with pytest.raises(ValueError):
        m.int8mm_block_forward(w, x[:, :128])
    m.int8mm_block_free(w)
    with pytest.raises(m.Int8mmError):
        m.int8mm_block_matmul(w, codes, scales)                   # freed


def test_empty_batches():
    w = m.int8mm_block_prepare_weight(acts(256, 64, F16, 2))
    x = torch.empty(0, 256, dtype=F16, device=dev())
    codes, scales = m.int8mm_block_quantize(x)
    assert codes.shape == (0, 256) and scales.shape == (0, 2)
    assert m.int8mm_block_matmul(w, codes, scales).shape == (0, 64)
    assert m.int8mm_block_forward(w, x).shape == (0, 64)
    assert m.int8mm_block_rms_norm(x, torch.ones(256, dtype=F16, device=dev()))[0].shape == (0, 256)


# -------------------------------------------------------------------- weight
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("K,N", [(16, 16), (128, 128), (144, 272), (1040, 784), (4096, 528), (65536, 32)])
def test_prepared_weight(K, N, dtype):
    W = acts(K, N, dtype, K + N)
    if K > 128:
        W[:128, :min(N, 128)] = 0  # a zero block
    w = m.int8mm_block_prepare_weight(W)
    codes, scales = m.int8mm_block_weight_codes(w)
    c, s = ref.quantise_blocks(W)
    same_quantised(codes, scales, c, s)
    w2 = m.int8mm_block_prepare_codes(codes, scales)
    codes2, scales2 = m.int8mm_block_weight_codes(w2)
    assert torch.equal(bits(codes), bits(codes2)) and torch.equal(scales, scales2)
    assert m.int8mm_block_weight_bytes(w) >= K * N


# ---------------------------------------------------------------------- norm
N_SHAPES = [(1, 16), (1, 12288), (2, 256), (5, 1040), (3, 65536), (129, 784), (300, 5120), (64, 4096), (9, 8208),
            (7, 32768), (3, 32784), (4000, 144)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("M,K", N_SHAPES)
def test_norm(M, K, dtype, with_residual):
    x = acts(M, K, dtype, M + K)
    r = acts(M, K, dtype, M + K + 1) if with_residual else None
    wt = (1 + 0.3 * torch.randn(K, generator=gen(K), device="cuda")).to(dtype)
    codes, scales, ro, y = m.int8mm_block_rms_norm(x, wt, 1e-5, residual=r, normed=True)
    h, y64 = ref.norm(x, r, wt, 1e-5)
    if with_residual:
        assert torch.equal(ro, h)
    else:
        assert ro is None
    ref.check_normed(y, y64)
    ref.check_quantised(codes, scales, y64)
    # each output alone is the same
    only_codes = m.int8mm_block_rms_norm(x, wt, 1e-5, residual=r)
    only_y = m.int8mm_block_rms_norm(x, wt, 1e-5, residual=r, codes=False, normed=True)
    assert torch.equal(bits(only_codes[0]), bits(codes)) and torch.equal(only_codes[1], scales)
    assert only_codes[3] is None and only_y[0] is None and torch.equal(only_y[3], y)


@pytest.mark.parametrize("onto", ["residual", "x"])
def test_norm_updates_the_residual_in_place(onto):
    x, r = acts(37, 1040, F16, 1), acts(37, 1040, F16, 2)
    wt = torch.ones(1040, dtype=F16, device=dev())
    want = m.int8mm_block_rms_norm(x, wt, residual=r)
    a, b = x.clone(), r.clone()
    out = b if onto == "residual" else a
    got = m.int8mm_block_rms_norm(a, wt, residual=b, residual_out=out)
    assert got[2] is out and torch.equal(out, want[2])
    assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1])
    with pytest.raises(m.Int8mmError):
        m.int8mm_block_rms_norm(a[:36], wt, residual=b[:36], residual_out=b[1:])


def test_norm_strided_rows_and_zero_rows():
    base = acts(40, 2048, BF16, 9)
    x, r = base[:, 16:1056], acts(40, 1056, BF16, 8)[:, 8:1048]
    base[3] = 0
    wt = torch.full((1040,), 0.5, dtype=BF16, device=dev())
    codes, scales, ro, y = m.int8mm_block_rms_norm(x, wt, 1e-6, residual=r, normed=True)
    h, y64 = ref.norm(x, r, wt, 1e-6)
    assert torch.equal(ro, h)
    ref.check_normed(y, y64)
    ref.check_quantised(codes, scales, y64)
    codes, scales, _, y = m.int8mm_block_rms_norm(x, wt, 1e-6, normed=True)
    assert (scales[3] == 0).all() and (codes[3].float() == 0).all() and (y[3] == 0).all()


def test_norm_a_bad_row_stays_alone():
    x = acts(8, 512, F16, 4)
    x[2, 7], x[5, 300] = float("nan"), float("inf")
    wt = torch.ones(512, dtype=F16, device=dev())
    codes, scales, _, y = m.int8mm_block_rms_norm(x, wt, normed=True)
    ok = torch.tensor([0, 1, 3, 4, 6, 7], device=dev())
    _, y64 = ref.norm(x, None, wt, 1e-6)
    ref.check_normed(y[ok], y64[ok])
    ref.check_quantised(codes[ok], scales[ok], y64[ok])
    assert y[2].isnan().all() and scales[2].isnan().all()
    # a row with Inf has the norm 0 everywhere but there, where it is NaN
    assert y[5, 300].isnan() and scales[5, 2].isnan()


# ------------------------------------------------------------------- product
P_SHAPES = [(1, 16, 16), (1, 128, 128), (1, 4096, 1040), (2, 144, 272), (16, 2048, 512), (17, 1040, 784),
            (33, 640, 4112), (37, 1040, 784), (64, 20480, 144), (65, 256, 256), (100, 512, 272), (128, 1024, 1024),
            (129, 1024, 1040), (200, 4096, 256), (256, 640, 512), (257, 1152, 528), (300, 1040, 784), (511, 272, 2064),
            (513, 640, 4112), (700, 2048, 1536), (1025, 400, 4112)]


def problem(M, K, N, dtype, seed, wide=False):
    x = acts(M, K, dtype, seed, wide)
    W = (torch.randn(K, N, generator=gen(seed + 1), device="cuda") * 0.02).to(dtype)
    w = m.int8mm_block_prepare_weight(W)
    codes, scales = m.int8mm_block_quantize(x)
    return x, w, codes, scales


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,N", P_SHAPES)
def test_product(M, K, N, dtype):
    x, w, codes, scales = problem(M, K, N, dtype, M + K + N)
    wc, ws = m.int8mm_block_weight_codes(w)
    bias = (torch.randn(N, generator=gen(7), device="cuda") * 0.5).to(dtype)
    y = m.int8mm_block_matmul(w, codes, scales, dtype=dtype)
    ref.check_product(y, codes, scales, wc, ws, None, K)
    yb = m.int8mm_block_matmul(w, codes, scales, bias=bias, dtype=dtype)
    ref.check_product(yb, codes, scales, wc, ws, bias, K)
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK
    # the same bits every time, and through the 16-bit entry point
    assert torch.equal(m.int8mm_block_matmul(w, codes, scales, dtype=dtype), y)
    assert torch.equal(m.int8mm_block_forward(w, x, bias=bias), yb)


@pytest.mark.parametrize("M", [1, 2, 9, 17, 33, 64])
@pytest.mark.parametrize("K,N", [(8192, 16384), (20480, 5120), (12288, 49152)])
def test_product_of_few_rows_over_many_tiles(M, K, N):
    """Runs of several tiles per cluster, tokens fewer than the CTAs that
    share the sums: the same bits every time, and no wait runs out."""
    x, w, codes, scales = problem(M, K, N, BF16, M + 1)
    y = m.int8mm_block_matmul(w, codes, scales, dtype=BF16)
    wc, ws = m.int8mm_block_weight_codes(w)
    cols = slice(0, 4096)
    ref.check_product(y[:, cols], codes, scales, wc[cols], ws[:32], None, K)
    ref.check_product(y[:, N - 4096:], codes, scales, wc[N - 4096:], ws[-32:], None, K)
    for _ in range(20):
        z = m.int8mm_block_matmul(w, codes, scales, dtype=BF16)
        assert torch.equal(y, z)
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK


def test_product_of_given_codes_of_every_kind():
    """All finite codes, scales over many magnitudes, zero blocks among them."""
    g = gen(11)
    for M, K, N in ((5, 400, 304), (200, 528, 272), (300, 1168, 400)):
        c = torch.randint(0, 256, (M, K), generator=g, device="cuda", dtype=torch.uint8)
        c = torch.where((c & 127) == 127, 0, c).view(torch.float8_e4m3fn)
        wc = torch.randint(0, 256, (N, K), generator=g, device="cuda", dtype=torch.uint8)
        wc = torch.where((wc & 127) == 127, 0, wc).view(torch.float8_e4m3fn)
        s = m.block._new_scales(M, ref.groups(K), dev())
        s.copy_(torch.ldexp(torch.ones(M, ref.groups(K), device="cuda"),
                            torch.randint(-30, -12, (M, ref.groups(K)), generator=g, device="cuda")))
        ws = torch.ldexp(torch.rand(ref.groups(N), ref.groups(K), generator=g, device="cuda"),
                         torch.randint(-10, 4, (ref.groups(N), ref.groups(K)), generator=g, device="cuda"))
        ws[0, 1] = 0
        s[2, 0] = 0
        w = m.int8mm_block_prepare_codes(wc, ws)
        for dtype in (F16, BF16):
            y = m.int8mm_block_matmul(w, c, s, dtype=dtype)
            ref.check_product(y, c, s, wc, ws, None, K)


@pytest.mark.parametrize("M", [3, 150, 300])
def test_product_nan_stays_in_its_row_and_overflow_is_inf(M):
    x, w, _, _ = problem(M, 512, 272, F16, 21)
    x[1, 500] = float("nan")
    x[2, 3] = float("inf")
    y = m.int8mm_block_forward(w, x)
    assert y[1].isnan().all() and y[2].isnan().all()
    keep = [i for i in range(M) if i not in (1, 2)]
    wc, ws = m.int8mm_block_weight_codes(w)
    codes, scales = m.int8mm_block_quantize(x)
    ref.check_product(y[keep], codes[keep], scales[keep], wc, ws, None, 512)
    big = m.int8mm_block_prepare_weight(torch.full((512, 272), 200.0, dtype=F16, device=dev()))
    z = m.int8mm_block_forward(big, torch.full((M, 512), 100.0, dtype=F16, device=dev()))
    assert (z == float("inf")).all()


@pytest.mark.parametrize("M", [1, 30, 100, 140, 300])
def test_product_writes_only_y_and_reads_no_scale_past_m(M):
    K, N, G = 1040, 784, 9
    x, w, codes, scales = problem(M, K, N, F16, 31)
    want = m.int8mm_block_matmul(w, codes, scales)
    # scales in a wider buffer, NaN between the groups' last rows and the next group
    lds = (M + 3) // 4 * 4 + 8
    wide = torch.full((G, lds), float("nan"), device=dev()).t()[:M]
    wide.copy_(scales)
    guard = 4096
    buf = torch.empty(2 * guard + M * N, dtype=F16, device=dev())
    buf.view(torch.int16).fill_(0x5a5a)
    Y = buf[guard:guard + M * N].view(M, N)
    m.int8mm_block_matmul(w, codes, wide, Y=Y)
    torch.cuda.synchronize()
    b = buf.view(torch.int16)
    assert (b[:guard] == 0x5a5a).all() and (b[guard + M * N:] == 0x5a5a).all()
    assert torch.equal(Y, want)


def test_quantise_and_norm_write_only_their_outputs():
    M, K = 37, 1040
    x, wt = acts(M, K, F16, 3), torch.ones(1040, dtype=F16, device=dev())
    want = m.int8mm_block_quantize(x)
    L, st = m.lib(), torch.cuda.current_stream().cuda_stream
    lds, G = 48, 9
    for norm in (False, True):
        c = torch.full((M * K + 8192,), 0x5a, dtype=torch.uint8, device=dev())
        s = torch.full((G * lds + 2048,), -7.0, device=dev())
        cp, sp = c.data_ptr() + 4096, s.data_ptr() + 4096
        if norm:
            q = m.int8mm_block_rms_norm(x, wt)
            assert L.int8mm_block_rms_norm(x.data_ptr(), K, None, 0, wt.data_ptr(), 0, M, K, 1e-6, None, None, cp, sp,
                                           lds, st) == 0
        else:
            q = want
            assert L.int8mm_block_quantize(x.data_ptr(), 0, M, K, K, cp, sp, lds, st) == 0
        torch.cuda.synchronize()
        assert (c[:4096] == 0x5a).all() and (c[4096 + M * K:] == 0x5a).all()
        assert torch.equal(c[4096:4096 + M * K].view(M, K), bits(q[0]))
        body = s[1024:1024 + G * lds].view(G, lds)
        assert torch.equal(body[:, :M].t(), q[1]) and (body[:, M:] == -7).all()
        assert (s[:1024] == -7).all() and (s[1024 + G * lds:] == -7).all()


@pytest.mark.parametrize("M", [5, 70, 300])
def test_forward_keeps_to_its_scratch(M):
    K, N = 1040, 784
    x, w, _, _ = problem(M, K, N, F16, 41)
    want = m.int8mm_block_forward(w, x)
    L, st = m.lib(), torch.cuda.current_stream().cuda_stream
    n = ctypes.c_size_t()
    assert L.int8mm_block_forward_scratch(w.handle, M, ctypes.byref(n)) == 0
    buf = torch.full((n.value + 8192,), 0x5a, dtype=torch.uint8, device=dev())
    Y = torch.zeros(M, N, dtype=F16, device=dev())

    def call(scratch=buf.data_ptr() + 4096, size=n.value, y=Y.data_ptr(), dtype=0, ldx=K):
        return L.int8mm_block_forward(w.handle, x.data_ptr(), ldx, M, None, y, dtype, scratch, size, st)

    assert call(size=n.value - 1) == m.INT8MM_ERR_INVALID_ARG
    assert call(scratch=None) == m.INT8MM_ERR_INVALID_ARG
    assert call(scratch=buf.data_ptr() + 4100) == m.INT8MM_ERR_ALIGNMENT
    assert call(scratch=x.data_ptr()) == m.INT8MM_ERR_INVALID_ARG
    assert call(y=buf.data_ptr() + 4096) == m.INT8MM_ERR_INVALID_ARG
    assert call(y=x.data_ptr()) == m.INT8MM_ERR_INVALID_ARG
    assert call(dtype=3) == m.INT8MM_ERR_INVALID_ARG
    assert call(ldx=K - 8) == m.INT8MM_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (buf == 0x5a).all() and (Y == 0).all()
    assert call() == 0
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and (buf[:4096] == 0x5a).all() and (buf[4096 + n.value:] == 0x5a).all()


# ----------------------------------------------------- streams, graphs, layers
def test_two_streams_share_a_handle():
    probs = [problem(M, 2048, 1040, F16, M) for M in (8, 100, 300, 8)]
    w = probs[0][1]
    want = [m.int8mm_block_matmul(w, c, s) for _, _, c, s in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [m.int8mm_block_matmul(w, c, s, stream=st) for st, (_, _, c, s) in zip(streams, probs)]
        got16 = [m.int8mm_block_forward(w, x, stream=st) for st, (x, _, _, _) in zip(streams, probs)]
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, got16):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_streams_by_handle_and_in_order():
    """A stream given as an integer; work queued behind slow work on it."""
    x, w, codes, scales = problem(40, 1040, 784, F16, 51)
    want = m.int8mm_block_forward(w, x)
    st = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(20):
            big = big @ big
            big /= big.norm()
        late.copy_(x)
    y = m.int8mm_block_forward(w, late, stream=st.cuda_stream)
    c, s = m.int8mm_block_quantize(late, stream=st.cuda_stream)
    z = m.int8mm_block_matmul(w, c, s, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want)


def test_host_threads_share_a_handle():
    x, w, _, _ = problem(33, 1040, 784, F16, 61)
    xs = [x, x[:1], acts(300, 1040, F16, 62), x[:20]]
    want = [m.int8mm_block_forward(w, v) for v in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(50):
                y = m.int8mm_block_forward(w, xs[i])
                try:
                    m.int8mm_block_forward(w, xs[i][:, :1024])  # refused, with this thread's message
                except ValueError:
                    pass
            st.synchronize()
            if not torch.equal(y, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_offsets_past_32_bits():
    """More than 2^32 values of X, 2^31 of Y; the last rows are right."""
    M, K = 66000, 65536
    x = torch.zeros(M, K, dtype=F16, device=dev())
    tail = acts(40, K, F16, 71)
    x[-40:] = tail
    codes, scales = m.int8mm_block_quantize(x)
    same_quantised(codes[-40:], scales[-40:], *ref.quantise(tail))
    assert (scales[:M - 40] == 0).all()
    del codes, scales
    wt = torch.ones(K, dtype=F16, device=dev())
    codes, scales, _, y = m.int8mm_block_rms_norm(x, wt, normed=True)
    one = m.int8mm_block_rms_norm(tail, wt, normed=True)
    assert torch.equal(bits(codes[-40:]), bits(one[0])) and torch.equal(scales[-40:], one[1])
    assert torch.equal(y[-40:], one[3])
    del x, y, codes, scales
    torch.cuda.empty_cache()
    M, K, N = 66000, 144, 32784
    x, w, codes, scales = problem(M, K, N, BF16, 72)
    y = m.int8mm_block_matmul(w, codes, scales, dtype=BF16)
    wc, ws = m.int8mm_block_weight_codes(w)
    for rows in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 5, M)):
        ref.check_product(y[rows], codes[rows], scales[rows], wc, ws, None, K)
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK


def test_a_weight_is_ready_for_the_work_queued_behind_it():
    """Preparation, norm and product back to back, with no wait between: each
    kernel may start while the last one ends, none may read early."""
    K, N, M = 4096, 4112, 300
    x = acts(M, K, F16, 1)
    wt = torch.ones(K, dtype=F16, device=dev())
    Ws = [(torch.randn(K, N, generator=gen(i), device="cuda") * 0.02).half() for i in range(6)]
    torch.cuda.synchronize()
    got = []
    for W in Ws:
        w = m.int8mm_block_prepare_weight(W)
        codes, scales, _, _ = m.int8mm_block_rms_norm(x, wt)
        got.append((w, codes, scales, m.int8mm_block_matmul(w, codes, scales), m.int8mm_block_forward(w, x[:9])))
    torch.cuda.synchronize()
    for w, codes, scales, y, few in got:
        assert torch.equal(m.int8mm_block_matmul(w, codes, scales), y)
        assert torch.equal(m.int8mm_block_forward(w, x[:9]), few)
        ref.check_product(y, codes, scales, *m.int8mm_block_weight_codes(w), None, K)


@pytest.mark.parametrize("M", [1, 40, 200, 600])
def test_captured_runs_replay_side_by_side(M):
    """Two graphs of norm, product, quantise and product over one set of
    weights, replayed at once on two streams with new inputs."""
    K, N = 1040, 2064
    w1 = m.int8mm_block_prepare_weight((torch.randn(K, N, generator=gen(1), device="cuda") * 0.02).half())
    w2 = m.int8mm_block_prepare_weight((torch.randn(N, K, generator=gen(2), device="cuda") * 0.02).half())
    wt = torch.ones(K, dtype=F16, device=dev())

    def step(x, r):
        codes, scales, ro, _ = m.int8mm_block_rms_norm(x, wt, residual=r)
        return m.int8mm_block_forward(w2, torch.relu(m.int8mm_block_matmul(w1, codes, scales))), ro

    xs = [acts(M, K, F16, 5 + i) for i in range(2)]
    rs = [acts(M, K, F16, 9 + i) for i in range(2)]
    step(xs[0], rs[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(xs[i], rs[i]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(3):
        for i in range(2):
            xs[i].copy_(acts(M, K, F16, 50 + 2 * k + i))
        torch.cuda.synchronize()
        for _ in range(4):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            y, ro = step(xs[i], rs[i])
            assert torch.equal(outs[i][0], y) and torch.equal(outs[i][1], ro)
    assert m.int8mm_block_get_status(w1) == m.INT8MM_OK and m.int8mm_block_get_status(w2) == m.INT8MM_OK


def test_layers_make_a_feed_forward_block():
    """norm -> expansion -> ReLU -> contraction, each step against its plain
    form on the step's own inputs; the 16-bit norm also feeds Linear8bitLt."""
    M, K, F = 75, 1040, 2064
    up, down = torch.nn.Linear(K, F).half().cuda(), torch.nn.Linear(F, K).half().cuda()
    norm = m.RMSNormBlock8bit(K)
    norm.weight.copy_((1 + 0.1 * torch.randn(K, generator=gen(3), device="cuda")).half())
    l1, l2 = m.LinearBlock8bit.from_linear(up), m.LinearBlock8bit.from_linear(down)
    x, r = acts(M, K, F16, 1).view(3, 25, K), acts(M, K, F16, 2).view(3, 25, K)
    (codes, scales), res = norm(x, r)
    h, y64 = ref.norm(x.view(M, K), r.view(M, K), norm.weight, norm.eps)
    assert res.shape == x.shape and torch.equal(res.view(M, K), h)
    ref.check_quantised(codes, scales, y64)
    a = l1((codes, scales))
    ref.check_product(a, codes, scales, *m.int8mm_block_weight_codes(l1._w), up.bias, K)
    a = torch.relu(a)
    out = l2(a.view(3, 25, F))
    assert out.shape == x.shape
    ref.check_product(out.view(M, K), *(t.cuda() for t in ref.quantise(a)), *m.int8mm_block_weight_codes(l2._w),
                      down.bias, F)
    y = m.int8mm_block_rms_norm(x.view(M, K), norm.weight.data, norm.eps, residual=r.view(M, K), codes=False,
                                normed=True)[3]
    lt = m.Linear8bitLt.from_linear(up)
    assert torch.equal(lt(y), m.int8mm_forward_bias(lt._w, y, 6.0, up.bias.detach()))
    pair = norm(x)
    assert isinstance(pair, tuple) and pair[0].shape == (M, K)


def test_the_wait_limit_has_a_floor():
    w = m.int8mm_block_prepare_weight(acts(256, 64, F16, 2))
    with pytest.raises(m.Int8mmError):
        m.int8mm_block_set_wait_limit(w, 999_999)
    m.int8mm_block_set_wait_limit(w, 1_000_000_000)
    assert m.int8mm_block_get_status(w) == m.INT8MM_OK
