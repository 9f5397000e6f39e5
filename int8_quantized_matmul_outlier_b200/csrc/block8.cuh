// The e4m3 block-scaled path: launchers and device helpers shared by its
// kernels.  Internal to libint8mm.so; the public C ABI is include/int8mm.h.
//
// A group is 128 consecutive columns of a row of activations (the last of a
// row may be short); a block is 128 x 128 of the weight.  Each has one fp32
// scale: value = code * scale, code an e4m3 number.
//
//   a = max |x| over the group, raised to 2^-100 if smaller and not 0
//   scale = a / 448,  code = e4m3(x * (448 / a)), both quotients and the
//   product rounded to fp32; a = 0 gives scale 0 and codes 0
//
// 448 is e4m3's largest number.  The floor 2^-100, which only bf16 data can
// go below, keeps 448 / a finite and a / 448 normal.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace i8mm {

constexpr int kGroup = 128;
constexpr float kE4m3Max = 448.0f;
constexpr float kGroupFloor = 7.888609052210118e-31f;  // 2^-100
constexpr int kDtypeF16 = 0, kDtypeBf16 = 1;

inline int64_t block_groups(int64_t k) { return (k + kGroup - 1) / kGroup; }

// ---- activations ----------------------------------------------------------
struct BlockRowArgs {
  const void* X;         // [M] rows of K 16-bit values, ldx apart
  int64_t M, K, ldx;
  const void* residual;  // norm: [M] rows, ldr apart, or nullptr
  int64_t ldr;
  const void* weight;    // norm: [K]
  float eps;
  void* residual_out;    // norm: [M, K] (may be X or residual itself), or nullptr
  void* normed;          // norm: [M, K] 16-bit, or nullptr
  uint8_t* codes;        // [M, K], or nullptr (norm only)
  float* scales;         // [G][lds]: group-major, rows lds apart
  int64_t lds;
};
cudaError_t launch_block_quantize(const BlockRowArgs& a, int dtype, cudaStream_t stream);
cudaError_t launch_block_rms_norm(const BlockRowArgs& a, int dtype, int num_sms, cudaStream_t stream);

// ---- weights (once per weight) --------------------------------------------
// Layout of the codes: Wb[g][n][128] with n < N_pad (a multiple of 256), rows
// past N and columns past K zero, so that the 128 x 128 operand tiles are
// contiguous.  Scales: sw[N / 128][G].
cudaError_t launch_block_weight_quantize(const void* W, int dtype, int64_t K, int64_t N, uint8_t* Wb, int64_t N_pad,
                                         float* sw, cudaStream_t stream);
cudaError_t launch_block_weight_pack(const uint8_t* codes, int64_t K, int64_t N, uint8_t* Wb, int64_t N_pad,
                                     cudaStream_t stream);
cudaError_t launch_block_weight_unpack(const uint8_t* Wb, int64_t K, int64_t N, int64_t N_pad, uint8_t* codes,
                                       cudaStream_t stream);

// ---- product ----------------------------------------------------------------
struct BlockGemmArgs {
  int M, N, K;
  int N_pad;             // rows per group in the weight layout
  const uint8_t* Wb;     // the codes of X and the scales sx come through tensor maps alone
  const float* sw;       // [N / 128][G]
  const void* bias;      // [N] of Y's type, or nullptr
  void* Y;               // [M, N]
  int bf16;              // Y's type
  int tiles, last_rows;  // few rows: the RowsPlan's
  int* status;           // device status word
  unsigned long long timeout_ns;
  int skip_scales;       // failure-detection tests only: one summing warp does not hand back its boxes of scales
  int skip_meeting;      // likewise, few rows: CTA 0 of a cluster does not count itself at the others' meeting
};

// Largest K of this path, as of the rest of the library.
constexpr int64_t kBlockMaxK = 65536;

#ifdef __CUDACC__
// Launch attribute that lets a kernel's blocks start while the stream's
// previous kernel finishes; returns 1, the number of attributes written.  The
// quantiser, the norm and the products are launched with it.  Every thread of
// theirs calls dependency_wait() before it reads or writes global memory: what
// ran before is then complete.  Ahead of it stands setup, and in the products a
// prefetch of weight tiles into L2, which returns no data and needs no order
// with their writer.  The kernels that prepare or read back a weight are
// launched without the attribute and without the wait.
inline unsigned overlap_attribute(cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  return 1;
}
__device__ __forceinline__ void dependency_wait() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------- device helpers
template <typename T>
__device__ __forceinline__ float2 pair_to_float(uint32_t w);
template <>
__device__ __forceinline__ float2 pair_to_float<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 pair_to_float<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t float_to_pair(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t float_to_pair<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t float_to_pair<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two floats to two e4m3 codes (round to nearest even, NaN to NaN), lo in the
// low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint2 e4m3_of8(const float (&v)[8], float r) {
  return make_uint2(e4m3_pair(__fmul_rn(v[0], r), __fmul_rn(v[1], r)) |
                        (e4m3_pair(__fmul_rn(v[2], r), __fmul_rn(v[3], r)) << 16),
                    e4m3_pair(__fmul_rn(v[4], r), __fmul_rn(v[5], r)) |
                        (e4m3_pair(__fmul_rn(v[6], r), __fmul_rn(v[7], r)) << 16));
}

// |x| of eight floats as bits, whose unsigned order is that of |x| with Inf
// and NaN above every number: a group that holds one gets it as its maximum.
__device__ __forceinline__ uint32_t absmax_bits8(const float (&v)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// The group's maximum to its scale and the factor 448 / a.  A NaN maximum
// gives NaN for both, Inf the scale Inf and the factor 0 (whose product with
// Inf is NaN): either way a product row that reads the group is NaN.
__device__ __forceinline__ void group_scale(uint32_t amax_bits, float& scale, float& factor) {
  float a = __uint_as_float(amax_bits);
  if (a < kGroupFloor && a > 0.0f) a = kGroupFloor;
  scale = __fdiv_rn(a, kE4m3Max);
  factor = a == 0.0f ? 0.0f : __fdiv_rn(kE4m3Max, a);
}
#endif

}  // namespace i8mm
