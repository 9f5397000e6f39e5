// Producers of e4m3 activations: the quantiser of 16-bit rows and the
// root-mean-square norm with the residual's addition (formulas in block8.cuh
// and at the kernels).  Both are bound by memory: every value is read once
// into registers and every output written once from there.
#include "block8.cuh"

namespace i8mm {
namespace {

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = pair_to_float<T>(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(float_to_pair<T>(v[0], v[1]), float_to_pair<T>(v[2], v[3]), float_to_pair<T>(v[4], v[5]),
                    float_to_pair<T>(v[6], v[7]));
}

template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), int64_t blocks, int threads, cudaStream_t stream, const A&... args) {
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = overlap_attribute(&attr);
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Maximum over the 16 lanes that hold a group.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// ------------------------------------------------------------- quantiser
// 16 lanes per group, 8 values per lane.  A warp takes a run of VPT * 4 groups
// of a row, all its loads before the first use: the bytes in flight per SM,
// not the arithmetic, set the rate.  Loads marked streaming, six blocks per SM
// (40 registers, 8 bytes of spills).  2048 x 20480 bf16, back to back over four
// inputs in turn: 4 vectors per lane 23.8 us, 2 26.8; with six blocks per SM
// 23.2, streaming 22.0 (5.7 TB/s).  Over three inputs in turn it takes 25 us.
constexpr int Q_THREADS = 256;

template <typename T, int VPT>
__global__ void __launch_bounds__(Q_THREADS, 6) block_quantize_kernel(const BlockRowArgs a, unsigned runs) {
  dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * (Q_THREADS / 32) + (threadIdx.x >> 5);
  const int64_t row = wid / runs;
  if (row >= a.M) return;
  const int nvec = static_cast<int>(a.K >> 3);
  const int c0 = static_cast<int>(wid - row * runs) * (VPT * 32) + lane;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(a.X) + row * a.ldx);
  uint4 u[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = c0 + j * 32;
    u[j] = c < nvec ? __ldcs(x + c) : make_uint4(0u, 0u, 0u, 0u);
  }
  uint2* codes = reinterpret_cast<uint2*>(a.codes + row * a.K);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = c0 + j * 32;
    float v[8], s, r;
    unpack8<T>(u[j], v);
    group_scale(max16(absmax_bits8(v)), s, r);
    if (c < nvec) {
      codes[c] = e4m3_of8(v, r);
      if ((lane & 15) == 0) a.scales[static_cast<int64_t>(c >> 4) * a.lds + row] = s;
    }
  }
}

// ------------------------------------------------------------------ norm
//   h = round16(x + residual)          (x itself without a residual)
//   y = h / sqrt(mean(h^2) + eps) * weight
// then residual_out = h, normed = round16(y), codes and scales of y (from
// fp32, not from its 16-bit rounding).  h is rounded before the norm because
// it is what the residual stream holds: the norm of residual_out alone gives
// the same y.  Bound by memory: 2048 x 12288 fp16 with a residual, back to back
// over four inputs in turn, takes 32 us, 5.5 TB/s of its 7 bytes per value (33.1
// with plain stores of residual_out; 512 threads per row 32.7, 128 threads 40);
// over three inputs in turn 35 us.  TPR threads hold a row in registers, VPT
// vectors of 8 values each; the sum of squares is fp32, in a fixed order.
template <typename T, int TPR, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS) block_rms_norm_kernel(const BlockRowArgs a) {
  constexpr int ROWS = THREADS / TPR, WPR = TPR / 32;
  __shared__ float part[THREADS / 32];
  dependency_wait();
  const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + rl;
  const bool row_ok = row < a.M;
  const int nvec = static_cast<int>(a.K >> 3);
  uint4 h[VPT];
  float sq = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = t + j * TPR;
    h[j] = make_uint4(0u, 0u, 0u, 0u);
    if (row_ok && c < nvec) h[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(a.X) + row * a.ldx) + c);
  }
  if (a.residual != nullptr) {
    const uint4* res = reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + row * a.ldr);
    constexpr int RB = TPR == 1024 && VPT > 4 ? 2 : VPT;  // residual vectors held at a time
#pragma unroll
    for (int j0 = 0; j0 < VPT; j0 += RB) {
      uint4 ru[RB];
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int c = t + (j0 + j) * TPR;
        if (row_ok && c < nvec) ru[j] = __ldcs(res + c);
      }
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int c = t + (j0 + j) * TPR;
        if (row_ok && c < nvec) {
          float x[8], r[8];
          unpack8<T>(h[j0 + j], x);
          unpack8<T>(ru[j], r);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(x[i], r[i]);
          h[j0 + j] = pack8<T>(x);
          // streaming: read much later
          __stcs(reinterpret_cast<uint4*>(static_cast<T*>(a.residual_out) + row * a.K) + c, h[j0 + j]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float x[8];
    unpack8<T>(h[j], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = __fmaf_rn(x[i], x[i], sq);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sq;
    __syncthreads();
    sq = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) sq += part[rl * WPR + w];
  }
  const float inv = __frsqrt_rn(__fadd_rn(__fdiv_rn(sq, static_cast<float>(a.K)), a.eps));
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = t + j * TPR;
    if (j * TPR >= nvec) break;  // the same for every thread
    const bool in = row_ok && c < nvec;
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
      float w[8];
      unpack8<T>(h[j], y);
      unpack8<T>(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(__fmul_rn(y[i], inv), w[i]);
      if (a.normed != nullptr) reinterpret_cast<uint4*>(static_cast<T*>(a.normed) + row * a.K)[c] = pack8<T>(y);
    }
    if (a.codes != nullptr) {
      float s, r;
      group_scale(max16(absmax_bits8(y)), s, r);
      if (in) {
        reinterpret_cast<uint2*>(a.codes + row * a.K)[c] = e4m3_of8(y, r);
        if ((t & 15) == 0) a.scales[static_cast<int64_t>(c >> 4) * a.lds + row] = s;
      }
    }
  }
}

template <typename T, int TPR, int VPT>
cudaError_t norm_t(const BlockRowArgs& a, cudaStream_t stream) {
  constexpr int THREADS = TPR < 128 ? 128 : TPR;
  constexpr int ROWS = THREADS / TPR;
  return launch_overlapped(block_rms_norm_kernel<T, TPR, VPT, THREADS>, (a.M + ROWS - 1) / ROWS, THREADS, stream, a);
}

// Threads per row and vectors per thread.  Few rows: as many threads as the
// row has vectors, up to 1024, for the shortest chain.  Many rows: 256 threads
// with up to 8 vectors each, so that several rows per SM are under way and
// one's loads run under another's sums and stores.  That ends at K = 16384:
// longer rows take 1024 threads and one or two rows are under way per SM (2048
// rows with a residual: K = 16384 50.6 us, 4.6 TB/s; 20480 71.9, 4.1; 32768
// 99.5, 4.7).  <1024, 8>, from K = 32784 on, spills 84 bytes.
template <typename T>
cudaError_t norm_d(const BlockRowArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t nvec = a.K / 8;
  if (nvec <= 32) return norm_t<T, 32, 1>(a, stream);
  if (a.M >= 2 * num_sms) {
    if (nvec <= 64) return norm_t<T, 32, 2>(a, stream);
    if (nvec <= 128) return norm_t<T, 32, 4>(a, stream);
    switch ((nvec + 255) / 256) {
      case 1: return norm_t<T, 256, 1>(a, stream);
      case 2: return norm_t<T, 256, 2>(a, stream);
      case 3: return norm_t<T, 256, 3>(a, stream);
      case 4: return norm_t<T, 256, 4>(a, stream);
      case 5: return norm_t<T, 256, 5>(a, stream);
      case 6: return norm_t<T, 256, 6>(a, stream);
      case 7: return norm_t<T, 256, 7>(a, stream);
      case 8: return norm_t<T, 256, 8>(a, stream);
    }
  }
  if (nvec <= 256) return norm_t<T, 256, 1>(a, stream);
  if (nvec <= 512) return norm_t<T, 512, 1>(a, stream);
  if (nvec <= 1024) return norm_t<T, 1024, 1>(a, stream);
  if (nvec <= 2048) return norm_t<T, 1024, 2>(a, stream);
  if (nvec <= 4096) return norm_t<T, 1024, 4>(a, stream);
  return norm_t<T, 1024, 8>(a, stream);
}

template <typename T>
cudaError_t quantize_d(const BlockRowArgs& a, cudaStream_t stream) {
  // runs of 4 vectors per lane; shorter ones for short rows, whose last run
  // would be mostly empty, and for few rows
  const int64_t nvec = a.K / 8;
  const int vpt = a.M * nvec < (1 << 18) ? 1 : (nvec % 128 == 0 || nvec >= 512 ? 4 : (nvec >= 192 ? 2 : 1));
  const unsigned runs = static_cast<unsigned>((nvec + vpt * 32 - 1) / (vpt * 32));
  const int64_t blocks = (a.M * runs + Q_THREADS / 32 - 1) / (Q_THREADS / 32);
  if (vpt == 4) return launch_overlapped(block_quantize_kernel<T, 4>, blocks, Q_THREADS, stream, a, runs);
  if (vpt == 2) return launch_overlapped(block_quantize_kernel<T, 2>, blocks, Q_THREADS, stream, a, runs);
  return launch_overlapped(block_quantize_kernel<T, 1>, blocks, Q_THREADS, stream, a, runs);
}

}  // namespace

cudaError_t launch_block_quantize(const BlockRowArgs& a, int dtype, cudaStream_t stream) {
  return dtype == kDtypeBf16 ? quantize_d<__nv_bfloat16>(a, stream) : quantize_d<__half>(a, stream);
}

cudaError_t launch_block_rms_norm(const BlockRowArgs& a, int dtype, int num_sms, cudaStream_t stream) {
  return dtype == kDtypeBf16 ? norm_d<__nv_bfloat16>(a, num_sms, stream) : norm_d<__half>(a, num_sms, stream);
}

}  // namespace i8mm
