// Layer norm of many rows, forward, that leaves x in 8 bits as well.
#include "flce_norm_stream_forward.cuh"

namespace flce {

cudaError_t launch_norm_stream_packed(const void* x, int bf16, int64_t ldx, const void* weight,
                                      const void* bias, int wbf16, int N, int D, float eps, void* y,
                                      int64_t ldy, float* mean, float* rstd, uint8_t* packed, int sms,
                                      cudaStream_t stream) {
  return launch_stream_forward<1>(x, bf16, ldx, weight, bias, wbf16, N, D, eps, y, ldy, mean, rstd, packed,
                                  sms, stream);
}

}  // namespace flce
