"""Life of e4m3 weight handles on the GPU: copies, saved and loaded layers,
freed handles, failed calls, host threads."""
import copy
import ctypes
import gc
import io
import pickle
import threading
import time
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import int8_quantized_matmul_outlier_b200 as m
from tests import _block8 as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def dev():
    return torch.device("cuda", torch.cuda.current_device())


def normal(*shape, seed, scale=1.0, dtype=F16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def layer(seed, K=272, N=144, dtype=F16, bias=True):
    w = m.int8mm_block_prepare_weight(normal(K, N, seed=seed, scale=0.02, dtype=dtype))
    return m.LinearBlock8bit(w, normal(N, seed=seed + 1, dtype=dtype) if bias else None, dtype)


# ---------------------------------------------------------------------- copies
@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy])
def test_a_dropped_copy_leaves_the_layer_alone(how):
    x = normal(5, 272, seed=1)
    a = layer(2)
    want = a(x)
    b = how(a)
    assert torch.equal(b(x), want)
    del b
    gc.collect()
    other = layer(3)  # takes what the copy may have given back
    assert torch.equal(a(x), want)
    del a
    gc.collect()
    assert other(x).shape == want.shape and m.int8mm_block_get_status(other._w) == m.INT8MM_OK


def test_a_pickled_layer_has_a_weight_of_its_own():
    x = normal(5, 272, seed=1)
    a = layer(2)
    want = a(x)
    b = pickle.loads(pickle.dumps(a))
    file = io.BytesIO()
    torch.save(a, file)
    file.seek(0)
    c = torch.load(file, weights_only=False)
    assert len({a._w.handle, b._w.handle, c._w.handle}) == 3
    m.int8mm_block_free(a._w)
    assert torch.equal(b(x), want) and torch.equal(c(x), want)
    with pytest.raises(m.Int8mmError):
        pickle.dumps(a)  # freed


# ------------------------------------------------------------------ saved state
@pytest.mark.parametrize("dtype,bias", [(F16, True), (BF16, False)])
def test_a_state_dict_holds_the_weight(dtype, bias):
    x = normal(5, 272, seed=1, dtype=dtype)
    a, b = (torch.nn.Sequential(torch.nn.Identity(), layer(s, dtype=dtype, bias=bias)) for s in (2, 9))
    want = a(x)
    assert not torch.equal(b(x), want)
    state = a.state_dict()
    assert set(state) == {"1.weight_codes", "1.weight_scales"} | ({"1.bias"} if bias else set())
    file = io.BytesIO()
    torch.save(state, file)
    file.seek(0)
    state = torch.load(file, map_location="cpu")
    b.load_state_dict(state)
    assert torch.equal(b(x), want)
    del a
    gc.collect()
    assert torch.equal(b(x), want)


def test_a_state_dict_that_does_not_fit_is_refused():
    a, x = layer(2), normal(5, 272, seed=1)
    want = a(x)
    good = a.state_dict()
    with pytest.raises(RuntimeError, match="Missing key.*weight_codes"):
        a.load_state_dict({"bias": good["bias"]})
    # (torch loads what fits before it raises: the bias is the layer's own)
    with pytest.raises(RuntimeError, match="weight_codes"):
        a.load_state_dict({**layer(3, K=288).state_dict(), "bias": good["bias"]})
    with pytest.raises(RuntimeError, match="scales"):
        a.load_state_dict({**good, "weight_scales": good["weight_scales"][:1]})
    with pytest.raises(RuntimeError, match="Unexpected key.*other"):
        a.load_state_dict({**good, "other": good["bias"]})
    assert torch.equal(a(x), want)
    assert a.load_state_dict({"bias": good["bias"]}, strict=False).missing_keys == ["weight_codes", "weight_scales"]
    assert torch.equal(a(x), want)


# --------------------------------------------------------------- freed handles
def test_a_freed_handle_stays_unknown():
    """A weight may lie where a freed one lay; the old handle does not name it."""
    L, n = m.lib(), ctypes.c_size_t()
    old = []
    for seed in range(8):
        w = layer(seed)._w
        for h in old:
            assert h != w.handle
            assert L.int8mm_block_weight_bytes(h, ctypes.byref(n)) == m.INT8MM_ERR_INVALID_ARG
            L.int8mm_block_free(h)  # no-op
        assert L.int8mm_block_weight_bytes(w.handle, ctypes.byref(n)) == m.INT8MM_OK
        old.append(w.handle)
        m.int8mm_block_free(w)


# ---------------------------------------------------------------- failed calls
def test_a_failed_preparation_leaves_no_error_behind():
    """Out of memory once; the next preparation, and the next launch outside
    the library, are not told of it."""
    big = torch.zeros(16384, 65536, dtype=F16, device=dev())  # its codes take 1 GB
    small, x = normal(256, 128, seed=1, scale=0.02), normal(3, 256, seed=2)
    torch.cuda.synchronize()
    fill = torch.empty(torch.cuda.mem_get_info()[0] - (600 << 20), dtype=torch.uint8, device=dev())
    for _ in range(2):
        with pytest.raises(m.Int8mmError) as e:
            m.int8mm_block_prepare_weight(big)
        assert e.value.status == m.INT8MM_ERR_OOM
    del fill, big
    torch.cuda.empty_cache()
    w = m.int8mm_block_prepare_weight(small)
    y = m.int8mm_block_forward(w, x)
    codes, scales = m.int8mm_block_quantize(x)
    ref.check_product(y, codes, scales, *m.int8mm_block_weight_codes(w), None, 256)


def test_no_preparation_on_a_captured_stream():
    """Refused, and the capture goes on."""
    W, x = normal(256, 128, seed=1, scale=0.02), normal(3, 256, seed=2)
    w = m.int8mm_block_prepare_weight(W)
    codes, scales = m.int8mm_block_weight_codes(w)
    want = m.int8mm_block_forward(w, x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = m.int8mm_block_forward(w, x)
        for prepare in (lambda: m.int8mm_block_prepare_weight(W), lambda: m.int8mm_block_prepare_codes(codes, scales)):
            with pytest.raises(m.Int8mmError) as e:
                prepare()
            assert e.value.status == m.INT8MM_ERR_INVALID_ARG
        z = m.int8mm_block_forward(w, x[:1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, m.int8mm_block_forward(w, x[:1]))


# ---------------------------------------------------------------- host threads
def test_host_threads_have_their_own_errors():
    """Products of one handle on a stream per thread, between calls that the
    library refuses; each thread reads its own message.  What fails in a thread
    fails the test."""
    K, N = 1040, 784
    w = m.int8mm_block_prepare_weight(normal(K, N, seed=1, scale=0.02))
    xs = [normal(M, K, seed=M) for M in (33, 1, 300, 20)]
    want = [m.int8mm_block_forward(w, x) for x in xs]
    torch.cuda.synchronize()
    L, start = m.lib(), threading.Barrier(len(xs))

    def work(i):
        st, ld = torch.cuda.Stream(), K - 8 * (i + 1)
        start.wait(timeout=60)
        for _ in range(100):
            y = m.int8mm_block_forward(w, xs[i], stream=st)
            assert L.int8mm_block_quantize(xs[i].data_ptr(), 0, xs[i].shape[0], K, ld, None, None, 4, None) == \
                m.INT8MM_ERR_INVALID_ARG
            time.sleep(0)  # another thread's turn
            assert f"row stride {ld} " in m.int8mm_last_error()
        st.synchronize()
        return torch.equal(y, want[i])

    with ThreadPoolExecutor(len(xs)) as pool:
        jobs = [pool.submit(work, i) for i in range(len(xs))]
        assert all(j.result(timeout=120) for j in jobs)


def test_the_default_stream_by_its_number():
    x, l = normal(5, 272, seed=1), layer(2, bias=False)
    want = l(x)
    assert torch.equal(m.int8mm_block_forward(l._w, x, stream=torch.cuda.default_stream().cuda_stream), want)
