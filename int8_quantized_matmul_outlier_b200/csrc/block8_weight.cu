// Preparation of an e4m3 block-scaled weight (once per weight): quantisation
// of a 16-bit W[K, N] by 128 x 128 blocks, or the layout change of codes that
// are given, into the group-blocked layout that the products read.  Both are
// one pass over the weight.
#include "block8.cuh"

namespace i8mm {
namespace {

// One thread block per 128 x 128 block of W.  Each thread holds 8 rows k of 8
// columns n; the codes go through shared memory to become n-major.
template <typename T>
__global__ void __launch_bounds__(256) block_weight_quantize_kernel(const T* W, int64_t K, int64_t N, uint8_t* Wb,
                                                                    int64_t N_pad, float* sw, int64_t G) {
  __shared__ __align__(16) uint8_t tile[128][128 + 16];  // [n][k], padded against bank conflicts
  __shared__ uint32_t amax_s[8];
  const int64_t g = blockIdx.x % G, nb = blockIdx.x / G;
  const int64_t k0 = g * kGroup, n0 = nb * kGroup;
  const int cn = (threadIdx.x & 15) * 8, ck = threadIdx.x >> 4;  // 8 columns; rows ck + 16 i
  float v[8][8];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t k = k0 + ck + 16 * i;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (k < K && n0 + cn < N) u = *reinterpret_cast<const uint4*>(W + k * N + n0 + cn);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 f = pair_to_float<T>(w[p]);
      v[i][2 * p] = f.x;
      v[i][2 * p + 1] = f.y;
    }
    m = max(m, absmax_bits8(v[i]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) amax_s[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, amax_s[w]);
  float s, r;
  group_scale(m, s, r);
  if (threadIdx.x == 0 && n0 < N) sw[nb * G + g] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint2 c = e4m3_of8(v[i], r);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[cn + j][ck + 16 * i] = static_cast<uint8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
  __syncthreads();
  uint8_t* dst = Wb + (g * N_pad + n0) * kGroup;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = threadIdx.x + 256 * i, n = e >> 3, c = (e & 7) * 16;
    *reinterpret_cast<uint4*>(dst + n * kGroup + c) = *reinterpret_cast<const uint4*>(&tile[n][c]);
  }
}

// codes [N, K] <-> Wb, 16 bytes per thread (K is a multiple of 16).
template <bool PACK>
__global__ void __launch_bounds__(256) block_weight_layout_kernel(uint8_t* codes, int64_t K, int64_t N, uint8_t* Wb,
                                                                  int64_t N_pad, int64_t G) {
  const int64_t total = G * (PACK ? N_pad : N) * 8;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * 256) {
    // n-major over the codes' rows, so that their side is contiguous
    const int64_t n = e / (G * 8), c = e - n * (G * 8);
    const int64_t g = c >> 3, k = c * 16;
    uint4* wb = reinterpret_cast<uint4*>(Wb + (g * N_pad + n) * kGroup + (c & 7) * 16);
    uint4* cd = reinterpret_cast<uint4*>(codes + n * K + k);
    if (PACK) *wb = (n < N && k < K) ? *cd : make_uint4(0u, 0u, 0u, 0u);
    else if (k < K) *cd = *wb;
  }
}

}  // namespace

cudaError_t launch_block_weight_quantize(const void* W, int dtype, int64_t K, int64_t N, uint8_t* Wb, int64_t N_pad,
                                         float* sw, cudaStream_t stream) {
  const int64_t G = block_groups(K);
  const unsigned grid = static_cast<unsigned>(G * (N_pad / kGroup));
  if (dtype == kDtypeBf16)
    block_weight_quantize_kernel<__nv_bfloat16>
        <<<grid, 256, 0, stream>>>(static_cast<const __nv_bfloat16*>(W), K, N, Wb, N_pad, sw, G);
  else
    block_weight_quantize_kernel<__half>
        <<<grid, 256, 0, stream>>>(static_cast<const __half*>(W), K, N, Wb, N_pad, sw, G);
  return cudaGetLastError();
}

cudaError_t launch_block_weight_pack(const uint8_t* codes, int64_t K, int64_t N, uint8_t* Wb, int64_t N_pad,
                                     cudaStream_t stream) {
  block_weight_layout_kernel<true>
      <<<2048, 256, 0, stream>>>(const_cast<uint8_t*>(codes), K, N, Wb, N_pad, block_groups(K));
  return cudaGetLastError();
}

cudaError_t launch_block_weight_unpack(const uint8_t* Wb, int64_t K, int64_t N, int64_t N_pad, uint8_t* codes,
                                       cudaStream_t stream) {
  block_weight_layout_kernel<false>
      <<<2048, 256, 0, stream>>>(codes, K, N, const_cast<uint8_t*>(Wb), N_pad, block_groups(K));
  return cudaGetLastError();
}

}  // namespace i8mm
