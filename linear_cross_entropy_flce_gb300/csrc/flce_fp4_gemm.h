// The product of two 4-bit matrices (flce_fp4_gemm.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace flce {

struct Fp4GemmParams {
  int N, V;                 // rows of H (tokens), rows of W
  int stages;               // of 256 values
  const uint8_t *h_scales, *w_scales;
  const float *h_rows, *w_rows;   // row scales, or null
  void* y;                  // [N][ldy], fp32 or bf16
  int64_t ldy;
  int64_t timeout_ns;
  int32_t* status;
};

// Rows of the tokens' tile for N tokens.
inline int fp4_tile(int64_t N) { return N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : N <= 128 ? 128 : 256; }

// y = H W^T. mW, mW32: W's codes in boxes of 128 bytes x 128 and x 32 rows; mH: H's in boxes of 128 bytes
// x kn rows, kn = fp4_tile(p.N).
cudaError_t launch_fp4_gemm(int kn, int nv, int bf16, const CUtensorMap& mW, const CUtensorMap& mW32,
                            const CUtensorMap& mH, const Fp4GemmParams& p, int sms, cudaStream_t stream);

}  // namespace flce
