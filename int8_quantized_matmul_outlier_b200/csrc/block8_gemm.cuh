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
}  // namespace i8mm
