// Layer norm over rows, forward and backward.
//
//   mean = sum x / D, rstd = 1 / sqrt(sum (x - mean)^2 / D + eps), h = (x - mean) rstd
//   y = h weight + bias
//   g = dy weight, dx = rstd (g - mean(g) - h mean(g h)),
//   dweight = sum_rows dy h, dbias = sum_rows dy
//
// One row per CTA; the row is read again (from the caches) for each of its passes. The
// sums over rows go through one fp32 partial per range of rows, joined in a fixed order.
#include <cmath>
#include <cstdint>

#include "flce_internal.h"

namespace flce {

namespace {

constexpr int kNormThreads = 256;
constexpr int kColumnThreads = 128;

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16)
              : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_from_f32(void* p, int64_t i, float v, int bf16) {
  if (bf16) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(v));
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(r & 0xFFFFu);
  } else {
    static_cast<float*>(p)[i] = v;
  }
}

// Sum of a pair over the block, the same value in every thread.
__device__ __forceinline__ float2 block_sum2(float2 v, float2* s_part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  __syncthreads();   // the sums of the call before have been read
  if (lane == 0) s_part[warp] = v;
  __syncthreads();
  float2 r = make_float2(0.f, 0.f);
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    r.x += s_part[w].x;
    r.y += s_part[w].y;
  }
  return r;
}

__global__ void __launch_bounds__(kNormThreads)
    layer_norm_kernel(const void* x, int bf16, int64_t ldx, const void* weight, const void* bias,
                      int wbf16, int N, int D, float eps, void* y, int64_t ldy, float* mean_out,
                      float* rstd_out) {
  __shared__ float2 s_part[kNormThreads / 32];
  for (int row = blockIdx.x; row < N; row += gridDim.x) {
    const int64_t xr = row * ldx, yr = row * ldy;
    float sum = 0.f;
    for (int i = threadIdx.x; i < D; i += kNormThreads) sum += load_as_f32(x, xr + i, bf16);
    const float mean = block_sum2(make_float2(sum, 0.f), s_part).x / D;
    float sq = 0.f;
    for (int i = threadIdx.x; i < D; i += kNormThreads) {
      const float d = load_as_f32(x, xr + i, bf16) - mean;
      sq = fmaf(d, d, sq);
    }
    const float rstd = 1.f / sqrtf(block_sum2(make_float2(sq, 0.f), s_part).x / D + eps);
    for (int i = threadIdx.x; i < D; i += kNormThreads) {
      const float h = (load_as_f32(x, xr + i, bf16) - mean) * rstd;
      const float w = weight != nullptr ? load_as_f32(weight, i, wbf16) : 1.f;
      const float b = bias != nullptr ? load_as_f32(bias, i, wbf16) : 0.f;
      store_from_f32(y, yr + i, fmaf(h, w, b), bf16);
    }
    if (threadIdx.x == 0) {
      if (mean_out != nullptr) mean_out[row] = mean;
      if (rstd_out != nullptr) rstd_out[row] = rstd;
    }
  }
}

__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dx_kernel(const void* dy, int64_t lddy, const void* x, int bf16, int64_t ldx,
                         const void* weight, int wbf16, const float* mean_in,
                         const float* rstd_in, int N, int D, void* dx, int64_t lddx) {
  __shared__ float2 s_part[kNormThreads / 32];
  for (int row = blockIdx.x; row < N; row += gridDim.x) {
    const int64_t xr = row * ldx, yr = row * lddy, gr = row * lddx;
    const float mean = mean_in[row], rstd = rstd_in[row];
    float2 sum = make_float2(0.f, 0.f);
    for (int i = threadIdx.x; i < D; i += kNormThreads) {
      const float w = weight != nullptr ? load_as_f32(weight, i, wbf16) : 1.f;
      const float g = load_as_f32(dy, yr + i, bf16) * w;
      sum.x += g;
      sum.y = fmaf(g, (load_as_f32(x, xr + i, bf16) - mean) * rstd, sum.y);
    }
    sum = block_sum2(sum, s_part);
    const float mg = sum.x / D, mgh = sum.y / D;
    for (int i = threadIdx.x; i < D; i += kNormThreads) {
      const float w = weight != nullptr ? load_as_f32(weight, i, wbf16) : 1.f;
      const float g = load_as_f32(dy, yr + i, bf16) * w;
      const float h = (load_as_f32(x, xr + i, bf16) - mean) * rstd;
      store_from_f32(dx, gr + i, rstd * (g - mg - h * mgh), bf16);
    }
  }
}

// Partial sums over a range of rows: part[range][0][i] = sum dy h, [1][i] = sum dy.
__global__ void __launch_bounds__(kColumnThreads)
    layer_norm_columns_kernel(const void* dy, int64_t lddy, const void* x, int bf16, int64_t ldx,
                              const float* mean, const float* rstd, int N, int D, int ranges,
                              float* part) {
  const int i = blockIdx.x * kColumnThreads + threadIdx.x;
  if (i >= D) return;
  const int range = blockIdx.y;
  float dw = 0.f, db = 0.f;
  for (int row = range; row < N; row += ranges) {
    const float d = load_as_f32(dy, row * lddy + i, bf16);
    dw = fmaf(d, (load_as_f32(x, row * ldx + i, bf16) - mean[row]) * rstd[row], dw);
    db += d;
  }
  part[(static_cast<int64_t>(range) * 2) * D + i] = dw;
  part[(static_cast<int64_t>(range) * 2 + 1) * D + i] = db;
}

__global__ void layer_norm_join_kernel(const float* __restrict__ part, int ranges, int D,
                                       void* dweight, void* dbias, int wbf16) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= D) return;
  float dw = 0.f, db = 0.f;
  for (int r = 0; r < ranges; ++r) {
    dw += part[(static_cast<int64_t>(r) * 2) * D + i];
    db += part[(static_cast<int64_t>(r) * 2 + 1) * D + i];
  }
  if (dweight != nullptr) store_from_f32(dweight, i, dw, wbf16);
  if (dbias != nullptr) store_from_f32(dbias, i, db, wbf16);
}

}  // namespace

cudaError_t launch_layer_norm(const void* x, int bf16, int64_t ldx, const void* weight,
                              const void* bias, int wbf16, int N, int D, float eps, void* y,
                              int64_t ldy, float* mean, float* rstd, int sms,
                              cudaStream_t stream) {
  const int grid = N < sms * 8 ? N : sms * 8;
  layer_norm_kernel<<<grid, kNormThreads, 0, stream>>>(x, bf16, ldx, weight, bias, wbf16, N, D,
                                                       eps, y, ldy, mean, rstd);
  return cudaGetLastError();
}

cudaError_t launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int bf16,
                                       int64_t ldx, const void* weight, int wbf16,
                                       const float* mean, const float* rstd, int N, int D,
                                       void* dx, int64_t lddx, void* dweight, void* dbias,
                                       float* part, int sms, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  // the column sums first: dx may overwrite dy
  if (dweight != nullptr || dbias != nullptr) {
    const int ranges = N < kNormRanges ? N : kNormRanges;
    const dim3 grid(static_cast<unsigned>((D + kColumnThreads - 1) / kColumnThreads),
                    static_cast<unsigned>(ranges));
    if (ranges > 0)
      layer_norm_columns_kernel<<<grid, kColumnThreads, 0, stream>>>(dy, lddy, x, bf16, ldx, mean,
                                                                     rstd, N, D, ranges, part);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    layer_norm_join_kernel<<<(D + 127) / 128, 128, 0, stream>>>(part, ranges, D, dweight, dbias,
                                                                wbf16);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (dx != nullptr && N > 0) {
    const int grid = N < sms * 8 ? N : sms * 8;
    layer_norm_dx_kernel<<<grid, kNormThreads, 0, stream>>>(dy, lddy, x, bf16, ldx, weight, wbf16,
                                                            mean, rstd, N, D, dx, lddx);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace flce
