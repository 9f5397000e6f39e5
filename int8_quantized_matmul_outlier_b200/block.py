"""The e4m3 block-scaled path: functions over the C ABI and two layers.

Activations are e4m3 codes [M, K] with one fp32 scale per 128 columns of a
row, weights e4m3 codes with one per 128 x 128 block; formulas, roundings and
edge rules are in ``include/int8mm.h``.  ``scales`` of activations is indexed
[M, G], G = ceil(K / 128), and stored group-major: strides (1, lds) with lds a
multiple of 4, as ``int8mm_block_quantize`` and ``int8mm_block_rms_norm``
return it.

Argument marshalling only, as in the package's other functions.  Work goes to
``stream``, or to the current stream of the arguments' device.
"""
from __future__ import annotations

import ctypes
import sys

import torch

from . import _P, _check, lib

_pkg = sys.modules[__package__]
GROUP = 128
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


def _groups(k: int) -> int:
    return -(-k // GROUP)


_fn = {}


def _c(name: str):
    """The C function of that name (looked up once: these calls are short)."""
    f = _fn.get(name)
    if f is None:
        f = _fn[name] = getattr(lib(), name)
    return f


def _here(device: torch.device, stream) -> bool:
    """Whether a call can run as it stands: on the current device's current stream."""
    return stream is None and device.index == torch._C._cuda_getDevice()


def _raw(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _elsewhere(fn, device: torch.device, stream, *args, **kw):
    """fn with `device` and `stream` made current: outputs allocated inside
    belong to the stream that writes them."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream is not None and stream.device != device:
        raise ValueError(f"stream on {stream.device}, arguments on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return fn(*args, **kw)


def _rows(t: torch.Tensor, name: str, like: torch.Tensor | None = None) -> int:
    """Checks a 2-D 16-bit CUDA tensor whose rows are contiguous (any row
    stride); its type's number."""
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float16 or bfloat16")
    if not (t.is_cuda and t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1)):
        raise ValueError(f"{name} must be a 2-D CUDA tensor with contiguous rows")
    if like is not None and (t.dtype != like.dtype or t.shape != like.shape or t.device != like.device):
        raise ValueError(f"{name} must have the shape, type and device of its companion")
    return d


def _ld(t: torch.Tensor) -> int:
    """Row stride; with one row any value will do, so the row's length."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _out(t: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _empty(rows: int, cols: int, dtype, device) -> torch.Tensor:
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)  # two thirds of torch.empty's time


def _new_scales(M: int, G: int, device) -> torch.Tensor:
    return torch.empty_strided((M, G), (1, (M + 3) // 4 * 4), dtype=torch.float32, device=device)


def _scales_ld(s: torch.Tensor, M: int, G: int, device) -> int:
    """The distance between the groups of scales [M, G]."""
    if s.dtype != torch.float32 or s.dim() != 2 or s.shape[0] != M or s.shape[1] != G or s.device != device:
        raise ValueError(f"scales must be float32 of shape ({M}, {G}) on {device}")
    if M == 0:
        return 4
    s0, lds = s.stride()
    if G == 1 and (lds < M or lds % 4 != 0):
        lds = (M + 3) // 4 * 4  # no second group to reach
    if (M > 1 and s0 != 1) or lds < M or lds % 4 != 0:
        raise ValueError("scales must be stored group-major: strides (1, lds), lds >= M a multiple of 4, "
                         "as int8mm_block_quantize returns it")
    return lds


class BlockWeight:
    """A prepared e4m3 weight with block scales (the library-owned handle).

    The weight never changes, so a copy, shallow or deep, is the object itself:
    the handle has one owner, and int8mm_block_free ends it for every holder.
    Pickling writes the codes and scales; loading prepares a weight from them."""

    def __init__(self, handle: int, K: int, N: int, device: torch.device):
        self.handle = handle
        self.K, self.N = K, N
        self.device = device

    def __copy__(self):
        return self

    def __deepcopy__(self, memo):
        return self

    def __reduce__(self):
        codes, scales = int8mm_block_weight_codes(self)
        return _from_bytes, (codes.view(torch.uint8), scales)  # plain pickle does not know the 8-bit type

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _pkg is not None and _pkg._lib is not None:  # at exit the module may be gone first
            _pkg._lib.int8mm_block_free(h)


def int8mm_block_prepare_weight(W: torch.Tensor, stream=None) -> BlockWeight:
    """Quantise a 16-bit weight W [K, N]; W is not kept."""
    if not (W.is_cuda and W.dim() == 2 and W.is_contiguous()):
        raise ValueError("W must be a contiguous 2-D CUDA tensor")
    dtype = _rows(W, "W")
    if not _here(W.device, stream):
        return _elsewhere(int8mm_block_prepare_weight, W.device, stream, W)
    out = _P()
    K, N = W.shape
    _check(_c("int8mm_block_prepare_weight")(W.data_ptr(), dtype, K, N, _raw(W.device), ctypes.byref(out)))
    return BlockWeight(out.value, K, N, W.device)


def int8mm_block_prepare_codes(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> BlockWeight:
    """A weight whose e4m3 codes [N, K] and scales [ceil(N/128), ceil(K/128)]
    (code * scale is the value) are at hand; neither is kept."""
    if not (codes.is_cuda and codes.dim() == 2 and codes.is_contiguous() and codes.dtype == torch.float8_e4m3fn):
        raise ValueError("codes must be a contiguous 2-D float8_e4m3fn CUDA tensor")
    N, K = codes.shape
    if (scales.dtype != torch.float32 or tuple(scales.shape) != (_groups(N), _groups(K))
            or scales.device != codes.device or not scales.is_contiguous()):
        raise ValueError(f"scales must be a contiguous float32 tensor [{_groups(N)}, {_groups(K)}] on codes' device")
    if not _here(codes.device, stream):
        return _elsewhere(int8mm_block_prepare_codes, codes.device, stream, codes, scales)
    out = _P()
    _check(_c("int8mm_block_prepare_codes")(codes.data_ptr(), scales.data_ptr(), K, N, _raw(codes.device),
                                            ctypes.byref(out)))
    return BlockWeight(out.value, K, N, codes.device)


def _from_bytes(codes: torch.Tensor, scales: torch.Tensor) -> BlockWeight:
    return int8mm_block_prepare_codes(codes.view(torch.float8_e4m3fn), scales)


def int8mm_block_weight_codes(w: BlockWeight, stream=None):
    """(codes [N, K] float8_e4m3fn, scales [ceil(N/128), ceil(K/128)] fp32) of a prepared weight."""
    if not _here(w.device, stream):
        return _elsewhere(int8mm_block_weight_codes, w.device, stream, w)
    codes = torch.empty((w.N, w.K), dtype=torch.float8_e4m3fn, device=w.device)
    scales = torch.empty((_groups(w.N), _groups(w.K)), dtype=torch.float32, device=w.device)
    _check(_c("int8mm_block_weight_codes")(w.handle, codes.data_ptr(), scales.data_ptr(), _raw(w.device)))
    return codes, scales


def int8mm_block_quantize(X: torch.Tensor, stream=None):
    """(codes [M, K] float8_e4m3fn, scales [M, G]) of 16-bit rows X [M, K]
    (rows contiguous, 16-byte aligned, any row stride)."""
    dtype, dev = _rows(X, "X"), X.device
    if not _here(dev, stream):
        return _elsewhere(int8mm_block_quantize, dev, stream, X)
    M, K = X.shape
    codes = _empty(M, K, torch.float8_e4m3fn, dev)
    lds = (M + 3) // 4 * 4
    scales = _new_scales(M, _groups(K), dev)
    st = _c("int8mm_block_quantize")(X.data_ptr(), dtype, M, K, _ld(X), codes.data_ptr(), scales.data_ptr(), lds,
                                     _raw(dev))
    if st:
        _check(st)
    return codes, scales


def int8mm_block_rms_norm(X: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                          residual: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                          codes: bool = True, normed: bool = False, stream=None):
    """Root-mean-square norm of X + residual, quantised: returns (codes [M, K],
    scales [M, G], residual_out [M, K], normed [M, K]), None for what is not
    asked for (``codes=False`` leaves out codes and scales, ``normed`` is the
    16-bit output) or has no residual.  ``residual_out`` may be ``residual`` or
    ``X`` itself, which is then updated in place."""
    dtype, dev = _rows(X, "X"), X.device
    M, K = X.shape
    if weight.dtype != X.dtype or weight.dim() != 1 or weight.shape[0] != K or weight.device != dev \
            or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous tensor of K elements of X's type on X's device")
    if residual is not None:
        _rows(residual, "residual", X)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if not (codes or normed):
        raise ValueError("neither codes nor the 16-bit output is asked for")
    if not _here(dev, stream):
        return _elsewhere(int8mm_block_rms_norm, dev, stream, X, weight, eps, residual, residual_out, codes, normed)
    ro = q = sc = y = ro_p = q_p = sc_p = y_p = res_p = None
    ldr, lds = K, (M + 3) // 4 * 4
    if residual is not None:
        ro = (_empty(M, K, X.dtype, dev) if residual_out is None
              else _out(residual_out, "residual_out", (M, K), X.dtype, dev))
        ro_p, res_p, ldr = ro.data_ptr(), residual.data_ptr(), _ld(residual)
    if codes:
        q = _empty(M, K, torch.float8_e4m3fn, dev)
        sc = _new_scales(M, _groups(K), dev)
        q_p, sc_p = q.data_ptr(), sc.data_ptr()
    if normed:
        y = _empty(M, K, X.dtype, dev)
        y_p = y.data_ptr()
    st = _c("int8mm_block_rms_norm")(X.data_ptr(), _ld(X), res_p, ldr, weight.data_ptr(), dtype, M, K, eps, ro_p, y_p,
                                     q_p, sc_p, lds, _raw(dev))
    if st:
        _check(st)
    return q, sc, ro, y


def _check_bias(bias: torch.Tensor | None, w: BlockWeight, dtype) -> None:
    if bias is not None and (bias.dtype != dtype or bias.numel() != w.N or not bias.is_contiguous()
                             or bias.device != w.device):
        raise ValueError("bias must be a contiguous tensor of N elements of Y's type on the weight's device")


def int8mm_block_matmul(w: BlockWeight, codes: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None,
                        Y: torch.Tensor | None = None, dtype: torch.dtype = torch.float16, stream=None) -> torch.Tensor:
    """Y [M, N] from activation codes [M, K] and scales [M, G]; ``dtype``
    (float16 or bfloat16) is Y's and the bias's type."""
    dev = w.device
    if codes.dtype != torch.float8_e4m3fn or not codes.is_cuda or codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous 2-D float8_e4m3fn CUDA tensor")
    M, K = codes.shape
    if K != w.K:
        raise ValueError(f"codes has {K} columns, the weight has K={w.K}")
    if codes.device != dev:
        raise ValueError(f"codes on {codes.device}, the weight on {dev}")
    d = _DTYPES.get(dtype)
    if d is None:
        raise ValueError("dtype must be float16 or bfloat16")
    lds = _scales_ld(scales, M, _groups(K), dev)
    _check_bias(bias, w, dtype)
    if not _here(dev, stream):
        return _elsewhere(int8mm_block_matmul, dev, stream, w, codes, scales, bias, Y, dtype)
    Y = _empty(M, w.N, dtype, dev) if Y is None else _out(Y, "Y", (M, w.N), dtype, dev)
    st = _c("int8mm_block_matmul")(w.handle, codes.data_ptr(), scales.data_ptr(), lds, M,
                                   None if bias is None else bias.data_ptr(), Y.data_ptr(), d, _raw(dev))
    if st:
        _check(st)
    return Y


def int8mm_block_forward(w: BlockWeight, X: torch.Tensor, bias: torch.Tensor | None = None,
                         Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Quantise 16-bit rows X [M, K] and multiply: Y [M, N] of X's type, the
    same as int8mm_block_quantize followed by int8mm_block_matmul."""
    d, dev = _rows(X, "X"), w.device
    M, K = X.shape
    if K != w.K:
        raise ValueError(f"X has {K} columns, the weight has K={w.K}")
    if X.device != dev:
        raise ValueError(f"X on {X.device}, the weight on {dev}")
    _check_bias(bias, w, X.dtype)
    if not _here(dev, stream):
        return _elsewhere(int8mm_block_forward, dev, stream, w, X, bias, Y)
    Y = _empty(M, w.N, X.dtype, dev) if Y is None else _out(Y, "Y", (M, w.N), X.dtype, dev)
    room = (M * K + 255) // 256 * 256 + (M + 3) // 4 * 16 * _groups(K)
    scratch = _empty(1, room, torch.uint8, dev)
    st = _c("int8mm_block_forward")(w.handle, X.data_ptr(), _ld(X), M, None if bias is None else bias.data_ptr(),
                                    Y.data_ptr(), d, scratch.data_ptr(), room, _raw(dev))
    if st:
        _check(st)
    return Y


def int8mm_block_get_status(w: BlockWeight) -> int:
    """Synchronises the device; returns the status code (does not raise)."""
    return int(lib().int8mm_block_get_status(w.handle))


def int8mm_block_set_wait_limit(w: BlockWeight, timeout_ns: int) -> None:
    """Limit of each device-side wait, in ns (at least 1e6)."""
    _check(lib().int8mm_block_set_wait_limit(w.handle, int(timeout_ns)))


INT8MM_BLOCK_TEST_SKIP_SCALES = 1
INT8MM_BLOCK_TEST_SKIP_MEETING = 2


def int8mm_block_set_test_skip(w: BlockWeight, bits: int) -> None:
    """Failure-detection tests only: later products leave out the arrivals
    named by `bits` (INT8MM_BLOCK_TEST_SKIP_*), so a device wait runs out."""
    _check(lib().int8mm_block_set_test_skip(w.handle, int(bits)))


def int8mm_block_weight_bytes(w: BlockWeight) -> int:
    n = ctypes.c_size_t()
    _check(lib().int8mm_block_weight_bytes(w.handle, ctypes.byref(n)))
    return int(n.value)


def int8mm_block_free(w: BlockWeight) -> None:
    h, w.handle = w.handle, None
    if h:
        lib().int8mm_block_free(h)


class LinearBlock8bit(torch.nn.Module):
    """y = x W + b with an e4m3 block-scaled weight, for inference.

    x is fp16 or bf16 [..., in_features], or a pair (codes, scales) as
    ``RMSNormBlock8bit`` and ``int8mm_block_quantize`` give it (the output is
    then [M, out_features] of ``dtype``).  The 16-bit weight is not kept.  The
    state dict holds the weight as ``weight_codes`` and ``weight_scales``;
    loading one prepares a new weight."""

    def __init__(self, weight: BlockWeight, bias: torch.Tensor | None = None, dtype: torch.dtype = torch.float16):
        super().__init__()
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float16 or bfloat16")
        self.in_features, self.out_features = weight.K, weight.N
        self.dtype = dtype
        self._w = weight
        self.bias = None if bias is None else torch.nn.Parameter(bias.to(dtype), requires_grad=False)

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear) -> "LinearBlock8bit":
        """The layer of an ``nn.Linear`` in fp16 or bf16 (whose weight is [out, in])."""
        with torch.no_grad():
            w = int8mm_block_prepare_weight(linear.weight.detach().t().contiguous())
            b = None if linear.bias is None else linear.bias.detach().clone()
        return cls(w, b, linear.weight.dtype)

    def _save_to_state_dict(self, destination, prefix, keep_vars):
        super()._save_to_state_dict(destination, prefix, keep_vars)
        destination[prefix + "weight_codes"], destination[prefix + "weight_scales"] = int8mm_block_weight_codes(self._w)

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys, unexpected_keys,
                              error_msgs):
        names = [prefix + "weight_codes", prefix + "weight_scales"]
        rest = {k: v for k, v in state_dict.items() if k not in names}
        super()._load_from_state_dict(rest, prefix, local_metadata, strict, missing_keys, unexpected_keys, error_msgs)
        missing_keys += [k for k in names if k not in state_dict]
        if any(k not in state_dict for k in names):
            return
        codes, scales = (state_dict[k] for k in names)
        if codes.dtype != torch.float8_e4m3fn or tuple(codes.shape) != (self.out_features, self.in_features):
            error_msgs.append(f"{names[0]}: {codes.dtype} {tuple(codes.shape)}, the layer takes torch.float8_e4m3fn "
                              f"{(self.out_features, self.in_features)}")
            return
        try:
            dev = self._w.device
            self._w = int8mm_block_prepare_codes(codes.to(dev).contiguous(), scales.to(dev).contiguous())
        except (ValueError, RuntimeError) as e:
            error_msgs.append(f"{names[0]}: {e}")

    def forward(self, x) -> torch.Tensor:
        if isinstance(x, tuple):
            codes, scales = x
            return int8mm_block_matmul(self._w, codes, scales, bias=self._bias(self.dtype), dtype=self.dtype)
        if x.shape[-1] != self.in_features:
            raise ValueError(f"last dimension {x.shape[-1]} != in_features {self.in_features}")
        y = int8mm_block_forward(self._w, x.reshape(-1, self.in_features), bias=self._bias(x.dtype))
        return y.reshape(*x.shape[:-1], self.out_features)

    def _bias(self, dtype):
        if self.bias is not None and self.bias.dtype != dtype:
            raise TypeError(f"activations of {dtype} with a bias of {self.bias.dtype}")
        return None if self.bias is None else self.bias.data

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}"


class RMSNormBlock8bit(torch.nn.Module):
    """Root-mean-square norm whose output is the (codes, scales) pair that
    ``LinearBlock8bit`` takes, for inference.

    ``forward(x)`` returns the pair; ``forward(x, residual)`` returns (pair, x +
    residual), with a residual of x's shape or one of the two as rows [M, dim].
    The pair of an x [..., dim] has one row per vector, codes [M, dim] and
    scales [M, G], whatever the leading dimensions; the sum keeps x's shape."""

    def __init__(self, dim: int, eps: float = 1e-6, dtype: torch.dtype = torch.float16, device=None):
        super().__init__()
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float16 or bfloat16")
        self.eps = float(eps)
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.weight = torch.nn.Parameter(torch.ones(dim, dtype=dtype, device=dev), requires_grad=False)

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        dim = self.weight.numel()
        if x.shape[-1] != dim:
            raise ValueError(f"last dimension {x.shape[-1]} != {dim}")
        if residual is not None and residual.shape != x.shape:
            ours, theirs = ([d for d in t.shape[:-1] if d != 1] for t in (x, residual))
            if ours != theirs and min(len(ours), len(theirs)) > 1:  # rows would meet in storage order
                raise ValueError(f"residual of shape {tuple(residual.shape)}, x of {tuple(x.shape)}")
        r = None if residual is None else residual.reshape(-1, dim)
        codes, scales, out, _ = int8mm_block_rms_norm(x.reshape(-1, dim), self.weight.data, self.eps, residual=r)
        return (codes, scales) if residual is None else ((codes, scales), out.reshape(x.shape))
