// Block-scaled formats (flce_pack.cu, flce_fp4.cu): layouts and launches.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace flce {

// ---- 8 bits: records of a row ---------------------------------------------------------

constexpr int kPackBlock = 32;

// Bytes of a row's codes, and of its record with the blocks' scale bytes behind them.
__host__ __device__ constexpr int64_t packed_codes(int64_t D) { return (D + 31) / 32 * 32; }
__host__ __device__ constexpr int64_t packed_record(int64_t D) {
  return packed_codes(D) + (packed_codes(D) / kPackBlock + 15) / 16 * 16;
}

cudaError_t launch_pack_e4m3(const void* x, int bf16, int64_t ldx, int N, int D, uint8_t* packed,
                             cudaStream_t stream);
cudaError_t launch_unpack_e4m3(const uint8_t* packed, int N, int D, void* x, int bf16, int64_t ldx,
                               cudaStream_t stream);

// Layer norm that leaves x packed, and its backward pass from that (bf16 / wbf16: types of the rows /
// of weight, bias and their gradients). part as launch_layer_norm_backward's.
cudaError_t launch_layer_norm_backward_packed(const void* dy, int64_t lddy, const uint8_t* packed, int bf16,
                                              const void* weight, int wbf16, const float* mean,
                                              const float* rstd, int N, int D, void* dx, int64_t lddx,
                                              void* dweight, void* dbias, float* part, int sms,
                                              cudaStream_t stream);

}  // namespace flce
