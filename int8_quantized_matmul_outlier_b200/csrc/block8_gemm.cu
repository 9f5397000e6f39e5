// Matrix product of e4m3 codes with block scales:
//   Y[m, n] = sum_g sx[g][m] sw[n / 128][g] sum_{k in g} X[m, k] W[n, k]  (+ bias[n])
// fp32 sums, one rounding to 16 bits.  A plain tiled kernel on the CUDA
// cores: 64 x 64 outputs per block, one group at a time in shared memory.
#include "block8.cuh"
#include "block8_gemm.cuh"

namespace i8mm {
namespace {

constexpr int T = 64;

__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float2 x = pair_to_float<__half>(lo), y = pair_to_float<__half>(hi);
  f[0] = x.x;
  f[1] = x.y;
  f[2] = y.x;
  f[3] = y.y;
}

template <typename TY>
__global__ void __launch_bounds__(256) block_gemm_simple_kernel(const BlockGemmArgs a) {
  __shared__ uint32_t xs[T][33], ws[T][33];
  const int m0 = blockIdx.y * T, n0 = blockIdx.x * T;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int G = (a.K + kGroup - 1) / kGroup;
  float acc[4][4] = {};
  for (int g = 0; g < G; ++g) {
    for (int e = threadIdx.x; e < T * 32; e += 256) {
      const int r = e >> 5, w = e & 31, k = g * kGroup + w * 4;
      xs[r][w] = (m0 + r < a.M && k < a.K)
                     ? *reinterpret_cast<const uint32_t*>(a.X + static_cast<size_t>(m0 + r) * a.K + k) : 0u;
      ws[r][w] = n0 + r < a.N_pad
                     ? *reinterpret_cast<const uint32_t*>(a.Wb + (static_cast<size_t>(g) * a.N_pad + n0 + r) * kGroup + w * 4)
                     : 0u;
    }
    __syncthreads();
    float part[4][4] = {};
    for (int w = 0; w < 32; ++w) {
      float x[4][4], y[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e4m3x4_to_float(xs[ty + 16 * i][w], x[i]);
        e4m3x4_to_float(ws[tx + 16 * i][w], y[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) part[i][j] = fmaf(x[i][k], y[j][k], part[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < a.M && n < a.N)
          acc[i][j] = fmaf(part[i][j], a.sx[static_cast<size_t>(g) * a.lds + m] * a.sw[(n / kGroup) * G + g], acc[i][j]);
      }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N) {
        float v = acc[i][j];
        if (a.bias != nullptr) v += static_cast<float>(static_cast<const TY*>(a.bias)[n]);
        static_cast<TY*>(a.Y)[static_cast<size_t>(m) * a.N + n] = TY(v);
      }
    }
}

}  // namespace

cudaError_t launch_block_gemm(const BlockGemmArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const dim3 grid((a.N + T - 1) / T, (a.M + T - 1) / T);
  if (a.bf16) block_gemm_simple_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
  else block_gemm_simple_kernel<__half><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace i8mm
