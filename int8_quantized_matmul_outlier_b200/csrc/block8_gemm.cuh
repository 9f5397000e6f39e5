// Launchers of the e4m3 block-scaled product (internal).
#pragma once
#include "block8.cuh"

namespace i8mm {

// Groups whose scales the kernel loads at a time.
constexpr int kSxChunk = 16;

// Columns of a tile of the CTA-pair kernel (rows: 256).
constexpr int kPairWidths[] = {256, 192, 160, 128};
int block_pair_width(int64_t M, int64_t N, int num_sms);
// tmX maps the codes [M, K] with 128-row boxes, tmW the weight's rows of 128
// bytes with width / 2-row boxes, tmS
// the scales [G][M] with 16 x 128 boxes.
cudaError_t launch_block_gemm_pair(const CUtensorMap& tmX, const CUtensorMap& tmW, const CUtensorMap& tmS,
                                   const BlockGemmArgs& a, int width, int num_sms, cudaStream_t stream);

// Few rows (M <= kRowsMaxM): clusters of `split` CTAs.
constexpr int64_t kRowsMaxM = 64;
struct RowsPlan {
  int split, clusters;
};
int rows_padded_tokens(int64_t M);
cudaError_t rows_max_clusters(int S, int* clusters);
RowsPlan rows_plan(int64_t N, int64_t K, const int (&max_clusters)[4]);  // for splits of 1, 2, 4, 8
// tmW and tmW16 map the weight's rows of 128 bytes with 128- and 16-row
// boxes, tmX the codes [M, K] with rows_padded_tokens(M)-row boxes, tmS the
// scales [G][M] with 16 x rows_padded_tokens(M) boxes.
cudaError_t launch_block_gemm_rows(const CUtensorMap& tmW, const CUtensorMap& tmW16, const CUtensorMap& tmX,
                                   const CUtensorMap& tmS, const BlockGemmArgs& a, const RowsPlan& p,
                                   cudaStream_t stream);
}  // namespace i8mm
