// Layer norm of many rows (flce_norm_stream*.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace flce {

// Whether the streaming kernels take rows of D elements of elt bytes: from 1 KB, so that a
// row's copy is worth its set-up, to what their rings hold.
bool norm_stream_fits(int D, int elt);

cudaError_t launch_norm_stream(const void* x, int bf16, int64_t ldx, const void* weight,
                               const void* bias, int wbf16, int N, int D, float eps, void* y,
                               int64_t ldy, float* mean, float* rstd, int sms,
                               cudaStream_t stream);

// dx, dweight, dbias may be null. *ranges partials are left in part ([ranges][2][D] floats),
// or dweight and dbias are done where *ranges is 1.
cudaError_t launch_norm_stream_backward(const void* dy, int64_t lddy, const void* x, int bf16,
                                        int64_t ldx, const void* weight, int wbf16,
                                        const float* mean, const float* rstd, int N, int D,
                                        void* dx, int64_t lddx, void* dweight, void* dbias,
                                        float* part, int* ranges, int sms, cudaStream_t stream);

// The forward pass that leaves x in 8 bits as well (of whole rows in registers, and of many), and the
// backward pass from that (flce_blocks.h).
cudaError_t launch_norm_pack(const void* x, int bf16, int64_t ldx, const void* weight, const void* bias,
                             int wbf16, int N, int D, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                             uint8_t* packed, cudaStream_t stream);
cudaError_t launch_norm_stream_packed(const void* x, int bf16, int64_t ldx, const void* weight,
                                      const void* bias, int wbf16, int N, int D, float eps, void* y,
                                      int64_t ldy, float* mean, float* rstd, uint8_t* packed, int sms,
                                      cudaStream_t stream);
cudaError_t launch_norm_stream_backward_packed(const void* dy, int64_t lddy, const uint8_t* packed, int bf16,
                                               const void* weight, int wbf16, const float* mean,
                                               const float* rstd, int N, int D, void* dx, int64_t lddx,
                                               void* dweight, void* dbias, float* part, int* ranges, int sms,
                                               cudaStream_t stream);

}  // namespace flce
