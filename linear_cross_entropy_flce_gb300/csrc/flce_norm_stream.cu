// Layer norm of many rows, forward.
#include "flce_norm_stream_forward.cuh"

namespace flce {

bool norm_stream_fits(int D, int elt) {
  const int row = D * elt;
  return row >= 1024 && row <= 16 * kStreamVectors * kForwardBlock;
}

cudaError_t launch_norm_stream(const void* x, int bf16, int64_t ldx, const void* weight,
                               const void* bias, int wbf16, int N, int D, float eps, void* y,
                               int64_t ldy, float* mean, float* rstd, int sms,
                               cudaStream_t stream) {
  return launch_stream_forward<0>(x, bf16, ldx, weight, bias, wbf16, N, D, eps, y, ldy, mean, rstd, nullptr,
                                  sms, stream);
}

}  // namespace flce
