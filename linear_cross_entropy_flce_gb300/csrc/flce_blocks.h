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

// ---- 4 bits -----------------------------------------------------------------------------
//
// Codes of a row: two to a byte, the first in the low bits, padded with zeros to whole 64s. Scale
// bytes as the tensor cores read them: for 128 rows and 4 neighbouring blocks of each, 512 bytes in which
// row r's four bytes are at (r % 32) * 16 + (r / 32) * 4; rows are padded to whole 128s and blocks to
// whole 256 values with zeros, the 512s of 128 rows follow one another.

constexpr int kFp4RowTile = 128;   // rows
constexpr int kFp4Stage = 256;     // values of a row

__host__ __device__ constexpr int fp4_block(int nv) { return nv ? 16 : 32; }
__host__ __device__ constexpr int64_t fp4_code_bytes(int64_t D) { return (D + 63) / 64 * 32; }
__host__ __device__ constexpr int64_t fp4_stages(int64_t D) { return (D + kFp4Stage - 1) / kFp4Stage; }
// Scale bytes of 128 rows' 256 values.
__host__ __device__ constexpr int fp4_stage_scales(int nv) { return kFp4RowTile * kFp4Stage / fp4_block(nv); }
__host__ __device__ constexpr int64_t fp4_scale_bytes(int64_t N, int64_t D, int nv) {
  return (N + kFp4RowTile - 1) / kFp4RowTile * fp4_stages(D) * fp4_stage_scales(nv);
}
// Where the four bytes of the blocks 4 q to 4 q + 3 of row r are.
__host__ __device__ constexpr int64_t fp4_scale_at(int64_t r, int64_t q, int64_t D, int nv) {
  return (r / kFp4RowTile * fp4_stages(D) * (fp4_stage_scales(nv) / 512) + q) * 512 + r % 32 * 16 +
         r % kFp4RowTile / 32 * 4;
}

// nv: nvfp4 (row_scales [N] fp32), else mxfp4 (null).
cudaError_t launch_quantize_fp4(const void* x, int bf16, int64_t ldx, int N, int D, int nv, uint8_t* codes,
                                uint8_t* scales, float* row_scales, cudaStream_t stream);
cudaError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* row_scales, int N,
                                  int D, int nv, void* x, int bf16, int64_t ldx, cudaStream_t stream);

cudaError_t launch_pack_e4m3(const void* x, int bf16, int64_t ldx, int N, int D, uint8_t* packed,
                             cudaStream_t stream);
cudaError_t launch_unpack_e4m3(const uint8_t* packed, int N, int D, void* x, int bf16, int64_t ldx,
                               cudaStream_t stream);

// Layer norm that leaves x packed, and its backward pass from that (bf16 / wbf16: types of the rows /
// of weight, bias and their gradients). part as launch_layer_norm_backward's.
cudaError_t launch_layer_norm_packed(const void* x, int bf16, int64_t ldx, const void* weight,
                                     const void* bias, int wbf16, int N, int D, float eps, void* y,
                                     int64_t ldy, float* mean, float* rstd, uint8_t* packed, int sms,
                                     cudaStream_t stream);
cudaError_t launch_layer_norm_backward_packed(const void* dy, int64_t lddy, const uint8_t* packed, int bf16,
                                              const void* weight, int wbf16, const float* mean,
                                              const float* rstd, int N, int D, void* dx, int64_t lddx,
                                              void* dweight, void* dbias, float* part, int sms,
                                              cudaStream_t stream);

}  // namespace flce
