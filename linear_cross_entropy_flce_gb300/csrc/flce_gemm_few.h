// Logits of a few tokens (flce_gemm_few.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "flce_gemm_params.h"

namespace flce {

constexpr int kFewPadRows = 128;   // rows of the padded copies of the tokens, all copies together

struct FewParams {
  int N, V, k_blocks;
  int copies;         // copies of the tokens that mH holds, kn rows each
  float* z;           // [N][ldz]
  int64_t ldz;
  int64_t timeout_ns;
  int32_t* status;
};

// Rows of the tokens' tile for N tokens.
inline int few_tile(int64_t N) { return N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : 128; }

// kFewPadRows rows of D: kFewPadRows / per copies of the N <= per tokens, padded with zeros.
cudaError_t launch_pad_tokens(const uint16_t* H, int N, int D, int per, uint16_t* out,
                              cudaStream_t stream);

// z = H W^T for p.N <= kn = few_tile(p.N) tokens.
cudaError_t launch_few_logits(int kn, const CUtensorMap& mW, const CUtensorMap& mW16,
                              const CUtensorMap& mH, const FewParams& p, int sms,
                              cudaStream_t stream);

}  // namespace flce
