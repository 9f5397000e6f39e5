// C ABI of the e4m3 block-scaled path (declared in include/int8mm.h): weight
// handles, argument checks and launches.  A handle holds the weight, its
// scales and a status word; every other buffer is the caller's, so calls on
// different streams and captured graphs share no workspace.
#include "block8.cuh"
#include "block8_gemm.cuh"
#include "int8mm.h"
#include "kernels.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <mutex>
#include <new>
#include <string>
#include <unordered_map>

using namespace i8mm;

struct int8mm_block_weight {
  int device = 0;
  int num_sms = 148;
  int64_t K = 0, N = 0, N_pad = 0;
  uint8_t* Wb = nullptr;  // [G][N_pad][128] codes
  float* sw = nullptr;    // [N / 128][G]
  int max_clusters[4] = {};  // of 1, 2, 4 and 8 CTAs, for products of few rows
  int* status = nullptr;
  unsigned long long timeout_ns = 2000000000ull;
  int test_skip = 0;  // INT8MM_BLOCK_TEST_SKIP_* bits (failure-detection tests only)
  size_t bytes = 0;
};

namespace {

// Callers hold a number in place of a pointer.  None is given twice, so a freed
// handle stays unknown when a later weight takes its memory.
std::mutex g_mu;
std::unordered_map<uintptr_t, int8mm_block_weight*> g_live;
uintptr_t g_last_handle = 0;

int8mm_status fail(int8mm_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int8mm_status fail(int8mm_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

// The runtime also keeps a failed call's error for the next one who asks, such
// as a launch of a later call, or of the caller: it is taken back here.
int8mm_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(e == cudaErrorMemoryAllocation ? INT8MM_ERR_OOM : INT8MM_ERR_CUDA, "%s: %s (%s)", what,
              cudaGetErrorName(e), cudaGetErrorString(e));
}

int8mm_block_weight* find(int8mm_block_weight_t handle) {
  std::lock_guard<std::mutex> g(g_mu);
  const auto at = g_live.find(reinterpret_cast<uintptr_t>(handle));
  return at == g_live.end() ? nullptr : at->second;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Makes a handle's device current for a call and puts the caller's back.
struct DeviceGuard {
  int prev = -1;
  cudaError_t err = cudaSuccess;
  explicit DeviceGuard(int dev) {
    err = cudaGetDevice(&prev);
    if (err == cudaSuccess && prev != dev) err = cudaSetDevice(dev);
    else prev = -1;
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

int sm_count() {
  static int cached[64] = {};
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return n;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  if (dev < 64) cached[dev] = n;
  return n;
}

int8mm_status check_dtype(int dtype) {
  if (dtype != INT8MM_DTYPE_FP16 && dtype != INT8MM_DTYPE_BF16)
    return fail(INT8MM_ERR_INVALID_ARG, "dtype %d: need INT8MM_DTYPE_FP16 or INT8MM_DTYPE_BF16", dtype);
  return INT8MM_OK;
}

int8mm_status check_k(int64_t K) {
  if (K < 16 || K % 16 != 0 || K > kBlockMaxK)
    return fail(INT8MM_ERR_UNSUPPORTED_SHAPE, "K=%lld: need a multiple of 16 in 16 .. %lld", (long long)K,
                (long long)kBlockMaxK);
  return INT8MM_OK;
}

int8mm_status check_m(int64_t M) {
  if (M < 0 || M >= (int64_t(1) << 31)) return fail(INT8MM_ERR_INVALID_ARG, "M=%lld out of range", (long long)M);
  return INT8MM_OK;
}

// 2-D array [rows, inner] (inner contiguous, rows `pitch` bytes apart), boxes
// of box_rows x box_inner, zero fill outside: bytes with the 128-byte swizzle,
// or floats without.
int8mm_status make_tmap(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows,
                        uint64_t pitch, uint32_t box_inner, uint32_t box_rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ok ? p : nullptr);
  }();
  if (fn == nullptr) return fail(INT8MM_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {inner, rows}, strides[1] = {pitch};
  const cuuint32_t box[2] = {box_inner, box_rows}, estr[2] = {1, 1};
  const CUresult r = fn(map, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? INT8MM_OK
                           : fail(INT8MM_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
}

// Rows of 16-bit values, ld apart.
int8mm_status check_rows(const char* name, const void* p, int64_t ld, int64_t K) {
  if (p == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "%s is NULL", name);
  if (ld < K || ld >= (int64_t(1) << 31))
    return fail(INT8MM_ERR_INVALID_ARG, "%s: row stride %lld with K=%lld", name, (long long)ld, (long long)K);
  if (!aligned16(p) || ld % 8 != 0)
    return fail(INT8MM_ERR_ALIGNMENT, "%s: rows must be 16-byte aligned (row stride %lld)", name, (long long)ld);
  return INT8MM_OK;
}

// (a TMA stride ends at 2^40 bytes)
int8mm_status check_scales(const float* scales, int64_t lds, int64_t M) {
  if (scales == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "scales is NULL");
  if (lds < M || lds % 4 != 0 || lds > (int64_t(1) << 32))
    return fail(INT8MM_ERR_INVALID_ARG,
                "scales: stride %lld between groups; need a multiple of 4 from M=%lld to 2^32", (long long)lds,
                (long long)M);
  if (!aligned16(scales)) return fail(INT8MM_ERR_ALIGNMENT, "scales must be 16-byte aligned");
  return INT8MM_OK;
}

struct Span {
  const char* name;
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr) return false;
  const auto pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + b.bytes && pb < pa + a.bytes;
}
int8mm_status check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlap(*o, i)) return fail(INT8MM_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
    for (auto q = outs.begin(); q != o; ++q)
      if (overlap(*o, *q)) return fail(INT8MM_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
  }
  return INT8MM_OK;
}
size_t rows_bytes(int64_t M, int64_t K, int64_t ld, size_t elem) {
  return static_cast<size_t>((M - 1) * ld + K) * elem;
}
size_t scales_bytes(int64_t M, int64_t K, int64_t lds) {
  if (M == 0) return 0;
  return static_cast<size_t>((block_groups(K) - 1) * lds + M) * 4;
}

// Layout of a forward's scratch: the codes, then the scales.
int64_t scales_ld(int64_t M) { return (M + 3) / 4 * 4; }
size_t codes_room(int64_t M, int64_t K) { return (static_cast<size_t>(M * K) + 255) / 256 * 256; }

void free_all(int8mm_block_weight* h) {
  if (h->Wb) cudaFree(h->Wb);
  if (h->sw) cudaFree(h->sw);
  if (h->status) cudaFree(h->status);
  delete h;
}

// Shared by the two ways to prepare a weight: from 16-bit W (scales NULL) or
// from codes and scales.
int8mm_status prepare(const void* W, int dtype, const float* scales, int64_t K, int64_t N, void* stream,
                      int8mm_block_weight_t* out) {
  if (out == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (W == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "W is NULL");
  int8mm_status st = check_k(K);
  if (st != INT8MM_OK) return st;
  if (N < 16 || N % 16 != 0 || N >= (int64_t(1) << 31) - 256)
    return fail(INT8MM_ERR_UNSUPPORTED_SHAPE, "N=%lld: need a multiple of 16, from 16", (long long)N);
  const int64_t N_pad = (N + kWeightRowPad - 1) / kWeightRowPad * kWeightRowPad;
  const int64_t G = block_groups(K);
  if (G * N_pad >= (int64_t(1) << 31))
    return fail(INT8MM_ERR_UNSUPPORTED_SHAPE, "K=%lld x N=%lld exceeds the weight layout's 2^31 rows of 128 bytes",
                (long long)K, (long long)N);
  if (!aligned16(W)) return fail(INT8MM_ERR_ALIGNMENT, "W must be 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // a captured allocation has no memory before the graph's launch, and new
  // memory at every launch; the handle would outlive neither
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (const cudaError_t e = cudaStreamIsCapturing(s, &capture); e != cudaSuccess) return cuda_fail(e, "stream query");
  if (capture != cudaStreamCaptureStatusNone)
    return fail(INT8MM_ERR_INVALID_ARG, "the stream is being captured: prepare weights before");
  int8mm_block_weight* h = new (std::nothrow) int8mm_block_weight();
  if (h == nullptr) return fail(INT8MM_ERR_OOM, "host allocation");
  cudaError_t e = cudaGetDevice(&h->device);
  h->num_sms = sm_count();
  h->K = K;
  h->N = N;
  h->N_pad = N_pad;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i) e = rows_max_clusters(1 << i, &h->max_clusters[i]);
  const size_t nsw = static_cast<size_t>((N + kGroup - 1) / kGroup * G);
  const size_t nwb = static_cast<size_t>(G * N_pad) * kGroup;
  if (e == cudaSuccess) e = cudaMallocAsync(reinterpret_cast<void**>(&h->Wb), nwb, s);
  if (e == cudaSuccess) e = cudaMallocAsync(reinterpret_cast<void**>(&h->sw), nsw * 4, s);
  if (e == cudaSuccess) e = cudaMallocAsync(reinterpret_cast<void**>(&h->status), 4, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->status, 0, 4, s);
  h->bytes = nwb + nsw * 4 + 4;
  if (e == cudaSuccess) {
    if (scales == nullptr) {
      e = launch_block_weight_quantize(W, dtype, K, N, h->Wb, N_pad, h->sw, s);
    } else {
      e = cudaMemcpyAsync(h->sw, scales, nsw * 4, cudaMemcpyDeviceToDevice, s);
      if (e == cudaSuccess) e = launch_block_weight_pack(static_cast<const uint8_t*>(W), K, N, h->Wb, N_pad, s);
    }
  }
  if (e != cudaSuccess) {
    cudaStreamSynchronize(s);
    free_all(h);
    return cuda_fail(e, "weight preparation");
  }
  try {
    std::lock_guard<std::mutex> g(g_mu);
    g_live.emplace(g_last_handle + 1, h);
    *out = reinterpret_cast<int8mm_block_weight_t>(++g_last_handle);
  } catch (const std::bad_alloc&) {
    cudaStreamSynchronize(s);
    free_all(h);
    return fail(INT8MM_ERR_OOM, "host allocation");
  }
  return INT8MM_OK;
}

}  // namespace

extern "C" {

int8mm_status int8mm_block_prepare_weight(const void* W_dev, int dtype, int64_t K, int64_t N, void* stream,
                                          int8mm_block_weight_t* out) {
  if (out != nullptr) *out = nullptr;
  int8mm_status st = check_dtype(dtype);
  return st != INT8MM_OK ? st : prepare(W_dev, dtype, nullptr, K, N, stream, out);
}

int8mm_status int8mm_block_prepare_codes(const void* codes_dev, const float* scales_dev, int64_t K, int64_t N,
                                         void* stream, int8mm_block_weight_t* out) {
  if (out != nullptr) *out = nullptr;
  if (scales_dev == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "scales is NULL");
  return prepare(codes_dev, 0, scales_dev, K, N, stream, out);
}

int8mm_status int8mm_block_weight_codes(int8mm_block_weight_t handle, void* codes_dev, float* scales_dev,
                                        void* stream) {
  int8mm_block_weight* h = find(handle);
  if (h == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "invalid or freed weight handle");
  if (codes_dev != nullptr && !aligned16(codes_dev)) return fail(INT8MM_ERR_ALIGNMENT, "codes must be 16-byte aligned");
  DeviceGuard dg(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = dg.err;
  if (e == cudaSuccess && codes_dev != nullptr)
    e = launch_block_weight_unpack(h->Wb, h->K, h->N, h->N_pad, static_cast<uint8_t*>(codes_dev), s);
  if (e == cudaSuccess && scales_dev != nullptr)
    e = cudaMemcpyAsync(scales_dev, h->sw, static_cast<size_t>((h->N + kGroup - 1) / kGroup * block_groups(h->K)) * 4,
                        cudaMemcpyDeviceToDevice, s);
  return e == cudaSuccess ? INT8MM_OK : cuda_fail(e, "weight read-back");
}

int8mm_status int8mm_block_quantize(const void* X_dev, int dtype, int64_t M, int64_t K, int64_t ldx, void* codes_dev,
                                    float* scales_dev, int64_t lds, void* stream) {
  int8mm_status st;
  if ((st = check_dtype(dtype)) != INT8MM_OK || (st = check_k(K)) != INT8MM_OK || (st = check_m(M)) != INT8MM_OK)
    return st;
  if (M == 0) return INT8MM_OK;
  if ((st = check_rows("X", X_dev, ldx, K)) != INT8MM_OK || (st = check_rows("codes", codes_dev, K, K)) != INT8MM_OK ||
      (st = check_scales(scales_dev, lds, M)) != INT8MM_OK ||
      (st = check_apart({{"codes", codes_dev, static_cast<size_t>(M * K)},
                         {"scales", scales_dev, scales_bytes(M, K, lds)}},
                        {{"X", X_dev, rows_bytes(M, K, ldx, 2)}})) != INT8MM_OK)
    return st;
  BlockRowArgs a = {};
  a.X = X_dev;
  a.M = M;
  a.K = K;
  a.ldx = ldx;
  a.codes = static_cast<uint8_t*>(codes_dev);
  a.scales = scales_dev;
  a.lds = lds;
  const cudaError_t e = launch_block_quantize(a, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? INT8MM_OK : cuda_fail(e, "quantiser launch");
}

int8mm_status int8mm_block_rms_norm(const void* X_dev, int64_t ldx, const void* residual_dev, int64_t ldr,
                                    const void* weight_dev, int dtype, int64_t M, int64_t K, float eps,
                                    void* residual_out_dev, void* normed_dev, void* codes_dev, float* scales_dev,
                                    int64_t lds, void* stream) {
  int8mm_status st;
  if ((st = check_dtype(dtype)) != INT8MM_OK || (st = check_k(K)) != INT8MM_OK || (st = check_m(M)) != INT8MM_OK)
    return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(INT8MM_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((residual_dev == nullptr) != (residual_out_dev == nullptr))
    return fail(INT8MM_ERR_INVALID_ARG, "residual and residual_out go together");
  if ((codes_dev == nullptr) != (scales_dev == nullptr))
    return fail(INT8MM_ERR_INVALID_ARG, "codes and scales go together");
  if (M == 0) return INT8MM_OK;
  if (codes_dev == nullptr && normed_dev == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "no output is asked for");
  const size_t out2 = static_cast<size_t>(M * K) * 2;
  if ((st = check_rows("X", X_dev, ldx, K)) != INT8MM_OK || (st = check_rows("weight", weight_dev, K, K)) != INT8MM_OK)
    return st;
  if (residual_dev != nullptr && ((st = check_rows("residual", residual_dev, ldr, K)) != INT8MM_OK ||
                                  (st = check_rows("residual_out", residual_out_dev, K, K)) != INT8MM_OK))
    return st;
  if (normed_dev != nullptr && (st = check_rows("normed", normed_dev, K, K)) != INT8MM_OK) return st;
  if (codes_dev != nullptr && ((st = check_rows("codes", codes_dev, K, K)) != INT8MM_OK ||
                               (st = check_scales(scales_dev, lds, M)) != INT8MM_OK))
    return st;
  const Span x = {"X", X_dev, rows_bytes(M, K, ldx, 2)}, w = {"weight", weight_dev, static_cast<size_t>(K) * 2};
  const Span r = {"residual", residual_dev, residual_dev ? rows_bytes(M, K, ldr, 2) : 0};
  const Span c = {"codes", codes_dev, static_cast<size_t>(M * K)};
  const Span sc = {"scales", scales_dev, codes_dev ? scales_bytes(M, K, lds) : 0};
  const Span no = {"normed", normed_dev, out2};
  // residual_out may be X or residual in place: each value is read before
  // the same thread writes it
  const bool on_x = residual_out_dev != nullptr && residual_out_dev == X_dev && ldx == K;
  const bool on_r = residual_out_dev != nullptr && residual_out_dev == residual_dev && ldr == K;
  const Span none = {"", nullptr, 0};
  if ((st = check_apart({c, sc, no}, {x, r, w})) != INT8MM_OK ||
      (st = check_apart({{"residual_out", residual_out_dev, out2}},
                        {on_x ? none : x, on_r ? none : r, w, c, sc, no})) != INT8MM_OK)
    return st;
  BlockRowArgs a = {};
  a.X = X_dev;
  a.M = M;
  a.K = K;
  a.ldx = ldx;
  a.residual = residual_dev;
  a.ldr = ldr;
  a.weight = weight_dev;
  a.eps = eps;
  a.residual_out = residual_out_dev;
  a.normed = normed_dev;
  a.codes = static_cast<uint8_t*>(codes_dev);
  a.scales = scales_dev;
  a.lds = lds;
  const cudaError_t e = launch_block_rms_norm(a, dtype, sm_count(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? INT8MM_OK : cuda_fail(e, "norm launch");
}

int8mm_status int8mm_block_matmul(int8mm_block_weight_t handle, const void* codes_dev, const float* scales_dev,
                                  int64_t lds, int64_t M, const void* bias_dev, void* Y_dev, int dtype,
                                  void* stream) {
  int8mm_block_weight* h = find(handle);
  if (h == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "invalid or freed weight handle");
  int8mm_status st;
  if ((st = check_dtype(dtype)) != INT8MM_OK || (st = check_m(M)) != INT8MM_OK) return st;
  if (M == 0) return INT8MM_OK;
  const int64_t K = h->K, N = h->N;
  if ((st = check_rows("codes", codes_dev, K, K)) != INT8MM_OK ||
      (st = check_scales(scales_dev, lds, M)) != INT8MM_OK || (st = check_rows("Y", Y_dev, N, N)) != INT8MM_OK)
    return st;
  if (bias_dev != nullptr && !aligned16(bias_dev)) return fail(INT8MM_ERR_ALIGNMENT, "bias must be 16-byte aligned");
  if (((M + 127) / 128) * ((N + 63) / 64) >= (int64_t(1) << 31))
    return fail(INT8MM_ERR_UNSUPPORTED_SHAPE, "M=%lld x N=%lld is too large", (long long)M, (long long)N);
  if ((st = check_apart({{"Y", Y_dev, static_cast<size_t>(M * N) * 2}},
                        {{"codes", codes_dev, static_cast<size_t>(M * K)},
                         {"scales", scales_dev, scales_bytes(M, K, lds)},
                         {"bias", bias_dev, static_cast<size_t>(N) * 2}})) != INT8MM_OK)
    return st;
  DeviceGuard dg(h->device);
  if (dg.err != cudaSuccess) return cuda_fail(dg.err, "cudaSetDevice");
  BlockGemmArgs a = {};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.N_pad = static_cast<int>(h->N_pad);
  a.Wb = h->Wb;
  a.sw = h->sw;
  a.bias = bias_dev;
  a.Y = Y_dev;
  a.bf16 = dtype == INT8MM_DTYPE_BF16;
  a.status = h->status;
  a.timeout_ns = h->timeout_ns;
  a.skip_scales = (h->test_skip & INT8MM_BLOCK_TEST_SKIP_SCALES) != 0;
  a.skip_meeting = (h->test_skip & INT8MM_BLOCK_TEST_SKIP_MEETING) != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool few = M <= kRowsMaxM;
  const int width = few ? 0 : block_pair_width(M, N, K, h->num_sms);
  const uint32_t box_m = few ? static_cast<uint32_t>(rows_padded_tokens(M)) : 128u;
  const uint64_t G = static_cast<uint64_t>(block_groups(K)), w_rows = G * static_cast<uint64_t>(h->N_pad);
  constexpr CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  CUtensorMap tmX, tmW, tmS, tmWl;
  if ((st = make_tmap(&tmX, u8, codes_dev, static_cast<uint64_t>(K), static_cast<uint64_t>(M),
                      static_cast<uint64_t>(K), kGroup, box_m)) != INT8MM_OK ||
      (st = make_tmap(&tmW, u8, h->Wb, kGroup, w_rows, kGroup, kGroup,
                      few ? 128u : static_cast<uint32_t>(width / 2))) != INT8MM_OK ||
      (st = make_tmap(&tmS, f32, scales_dev, static_cast<uint64_t>(M), G, static_cast<uint64_t>(lds) * 4, box_m,
                      kSxChunk)) != INT8MM_OK)
    return st;
  cudaError_t e;
  if (few) {
    const RowsPlan plan = rows_plan(M, N, K, h->max_clusters);
    if ((st = make_tmap(&tmWl, u8, h->Wb, kGroup, w_rows, kGroup, kGroup,
                        static_cast<uint32_t>(plan.last_rows))) != INT8MM_OK)
      return st;
    a.tiles = plan.tiles;
    a.last_rows = plan.last_rows;
    e = launch_block_gemm_rows(tmW, tmWl, tmX, tmS, a, plan, s);
  } else {
    e = launch_block_gemm_pair(tmX, tmW, tmS, a, width, h->num_sms, s);
  }
  return e == cudaSuccess ? INT8MM_OK : cuda_fail(e, "block-scaled product launch");
}

int8mm_status int8mm_block_forward_scratch(int8mm_block_weight_t handle, int64_t M, size_t* bytes) {
  const int8mm_block_weight* h = find(handle);
  if (h == nullptr || bytes == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "invalid handle or NULL output");
  const int8mm_status st = check_m(M);
  if (st == INT8MM_OK) *bytes = codes_room(M, h->K) + scales_bytes(scales_ld(M), h->K, scales_ld(M));
  return st;
}

int8mm_status int8mm_block_forward(int8mm_block_weight_t handle, const void* X_dev, int64_t ldx, int64_t M,
                                   const void* bias_dev, void* Y_dev, int dtype, void* scratch_dev,
                                   size_t scratch_bytes, void* stream) {
  size_t need = 0;
  int8mm_status st = int8mm_block_forward_scratch(handle, M, &need);
  if (st != INT8MM_OK || (st = check_dtype(dtype)) != INT8MM_OK) return st;
  if (M == 0) return INT8MM_OK;
  const int8mm_block_weight* h = find(handle);
  if (h == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "invalid or freed weight handle");
  if (scratch_dev == nullptr || scratch_bytes < need)
    return fail(INT8MM_ERR_INVALID_ARG, "scratch of %zu bytes: need %zu", scratch_dev ? scratch_bytes : 0, need);
  if (!aligned16(scratch_dev)) return fail(INT8MM_ERR_ALIGNMENT, "scratch must be 16-byte aligned");
  if ((st = check_rows("X", X_dev, ldx, h->K)) != INT8MM_OK || (st = check_rows("Y", Y_dev, h->N, h->N)) != INT8MM_OK)
    return st;
  if (bias_dev != nullptr && !aligned16(bias_dev)) return fail(INT8MM_ERR_ALIGNMENT, "bias must be 16-byte aligned");
  // Y may lie on neither X nor the scratch; the two steps check the rest
  if ((st = check_apart({{"Y", Y_dev, static_cast<size_t>(M * h->N) * 2}, {"scratch", scratch_dev, need}},
                        {{"X", X_dev, rows_bytes(M, h->K, ldx, 2)},
                         {"bias", bias_dev, static_cast<size_t>(h->N) * 2}})) != INT8MM_OK)
    return st;
  DeviceGuard dg(h->device);
  if (dg.err != cudaSuccess) return cuda_fail(dg.err, "cudaSetDevice");
  float* scales = reinterpret_cast<float*>(static_cast<char*>(scratch_dev) + codes_room(M, h->K));
  st = int8mm_block_quantize(X_dev, dtype, M, h->K, ldx, scratch_dev, scales, scales_ld(M), stream);
  if (st != INT8MM_OK) return st;
  return int8mm_block_matmul(handle, scratch_dev, scales, scales_ld(M), M, bias_dev, Y_dev, dtype, stream);
}

int8mm_status int8mm_block_get_status(int8mm_block_weight_t handle) {
  int8mm_block_weight* h = find(handle);
  if (h == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "invalid or freed weight handle");
  DeviceGuard dg(h->device);
  cudaError_t e = dg.err;
  int word = 0;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&word, h->status, 4, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, 4);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  return (word & kStatusTimeout) ? fail(INT8MM_ERR_TIMEOUT, "a device wait ran out of time") : INT8MM_OK;
}

int8mm_status int8mm_block_set_wait_limit(int8mm_block_weight_t handle, uint64_t timeout_ns) {
  int8mm_block_weight* h = find(handle);
  if (h == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "invalid or freed weight handle");
  if (timeout_ns < 1000000ull)
    return fail(INT8MM_ERR_INVALID_ARG, "timeout %llu ns is below the 1 ms minimum",
                static_cast<unsigned long long>(timeout_ns));
  h->timeout_ns = timeout_ns;
  return INT8MM_OK;
}

int8mm_status int8mm_block_set_test_skip(int8mm_block_weight_t handle, int bits) {
  int8mm_block_weight* h = find(handle);
  if (h == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "invalid or freed weight handle");
  if ((bits & ~(INT8MM_BLOCK_TEST_SKIP_SCALES | INT8MM_BLOCK_TEST_SKIP_MEETING)) != 0)
    return fail(INT8MM_ERR_INVALID_ARG, "unknown test bits 0x%x", bits);
  h->test_skip = bits;
  return INT8MM_OK;
}

int8mm_status int8mm_block_weight_bytes(int8mm_block_weight_t handle, size_t* bytes) {
  const int8mm_block_weight* h = find(handle);
  if (h == nullptr || bytes == nullptr) return fail(INT8MM_ERR_INVALID_ARG, "invalid handle or NULL output");
  *bytes = h->bytes;
  return INT8MM_OK;
}

void int8mm_block_free(int8mm_block_weight_t handle) {
  int8mm_block_weight* h = nullptr;
  {
    std::lock_guard<std::mutex> g(g_mu);
    const auto at = g_live.find(reinterpret_cast<uintptr_t>(handle));
    if (at == g_live.end()) return;
    h = at->second;
    g_live.erase(at);
  }
  DeviceGuard dg(h->device);
  cudaDeviceSynchronize();
  free_all(h);
}

}  // extern "C"
