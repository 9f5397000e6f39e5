// Launchers of the e4m3 block-scaled product (internal).
#pragma once
#include <atomic>

#include "block8.cuh"

namespace i8mm {

// Allows a kernel its dynamic shared memory, once per device (of the first 64;
// on others every time).
template <typename F>
cudaError_t smem_attribute_once(F kern, int bytes, std::atomic<unsigned long long>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Groups whose scales the kernel loads at a time.
constexpr int kSxChunk = 16;

// Columns of a tile of the CTA-pair kernel (rows: 256): 256 or 128.
int block_pair_width(int64_t M, int64_t N, int64_t K, int num_sms);
// tmX maps the codes [M, K] with 128-row boxes, tmW the weight's rows of 128
// bytes with width / 2-row boxes, tmS
// the scales [G][M] with 16 x 128 boxes.
cudaError_t launch_block_gemm_pair(const CUtensorMap& tmX, const CUtensorMap& tmW, const CUtensorMap& tmS,
                                   const BlockGemmArgs& a, int width, int num_sms, cudaStream_t stream);

// Few rows (M <= kRowsMaxM): clusters of `split` CTAs.
constexpr int64_t kRowsMaxM = 64;
struct RowsPlan {
  int split, clusters;   // CTAs of a cluster, clusters
  int tiles, last_rows;  // of the longest run: tiles, rows of the last one
};
int rows_padded_tokens(int64_t M);
cudaError_t rows_max_clusters(int S, int* clusters);
RowsPlan rows_plan(int64_t M, int64_t N, int64_t K, const int (&max_clusters)[4]);  // for splits of 1, 2, 4, 8
// tmW and tmWl map the weight's rows of 128 bytes with 128- and
// p.last_rows-row boxes (a.tiles and a.last_rows are p's), tmX the codes
// [M, K] with rows_padded_tokens(M)-row boxes, tmS the scales [G][M] with 16 x
// rows_padded_tokens(M) boxes.
cudaError_t launch_block_gemm_rows(const CUtensorMap& tmW, const CUtensorMap& tmWl, const CUtensorMap& tmX,
                                   const CUtensorMap& tmS, const BlockGemmArgs& a, const RowsPlan& p,
                                   cudaStream_t stream);
}  // namespace i8mm
