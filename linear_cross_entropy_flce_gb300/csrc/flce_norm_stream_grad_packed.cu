// Layer norm of many rows, backward, from x kept in 8 bits.
#include "flce_norm_stream_grad.cuh"

namespace flce {

cudaError_t launch_norm_stream_backward_packed(const void* dy, int64_t lddy, const uint8_t* packed, int bf16,
                                               const void* weight, int wbf16, const float* mean,
                                               const float* rstd, int N, int D, void* dx, int64_t lddx,
                                               void* dweight, void* dbias, float* part, int* ranges, int sms,
                                               cudaStream_t stream) {
  return launch_stream_grad<1>(dy, lddy, packed, bf16, packed_record(D), weight, wbf16, mean, rstd, N, D, dx,
                               lddx, dweight, dbias, part, ranges, sms, stream);
}

}  // namespace flce
