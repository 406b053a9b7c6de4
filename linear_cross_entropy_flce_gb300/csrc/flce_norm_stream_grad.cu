// Layer norm of many rows, backward, from x.
#include "flce_norm_stream_grad.cuh"

namespace flce {

cudaError_t launch_norm_stream_backward(const void* dy, int64_t lddy, const void* x, int bf16,
                                        int64_t ldx, const void* weight, int wbf16,
                                        const float* mean, const float* rstd, int N, int D,
                                        void* dx, int64_t lddx, void* dweight, void* dbias,
                                        float* part, int* ranges, int sms, cudaStream_t stream) {
  return launch_stream_grad<0>(dy, lddy, x, bf16, ldx, weight, wbf16, mean, rstd, N, D, dx, lddx, dweight,
                               dbias, part, ranges, sms, stream);
}

}  // namespace flce
