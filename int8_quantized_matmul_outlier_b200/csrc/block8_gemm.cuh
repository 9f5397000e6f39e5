// Launchers of the e4m3 block-scaled product (internal).
#pragma once
#include "block8.cuh"

namespace i8mm {
cudaError_t launch_block_gemm(const BlockGemmArgs& a, int num_sms, cudaStream_t stream);
}  // namespace i8mm
