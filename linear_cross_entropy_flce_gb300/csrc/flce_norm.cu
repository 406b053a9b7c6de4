// Layer norm over rows, forward and backward.
//
//   mean = sum x / D, rstd = 1 / sqrt(sum (x - mean)^2 / D + eps), h = (x - mean) rstd
//   y = h weight + bias
//   g = dy weight, dx = rstd (g - mean(g) - h mean(g h)),
//   dweight = sum_rows dy h, dbias = sum_rows dy
//
// Forward: a group of R threads holds a row in registers, so it is read once; the variance
// is taken from centred values. Backward: the groups of a persistent grid walk the rows,
// each thread owning the same columns of every row, so that dweight and dbias accumulate
// in its registers while dx is formed from the same loads; the next row is loaded before
// the current one is reduced. One fp32 partial per CTA is left, joined in a fixed order. These
// serve few and short rows, where latency counts: 1 x 4096 bf16 2.9 us forward and 8.0
// backward, 16384 x 128 6.0 and 12.1.
//
// Many rows of 1 KB or more go through the kernels of flce_norm_stream*.cu instead.
//
// Accesses are as wide as the hidden size, the strides and the addresses allow (VW
// elements, 2 to 16 bytes). Rows longer than 1024 threads can hold take the looped
// kernels, which read a row again for each of its passes.
#include <cmath>
#include <cstdint>

#include "flce_internal.h"
#include "flce_launch.cuh"
#include "flce_norm.cuh"
#include "flce_norm_stream.h"

namespace flce {

namespace {

constexpr int kNormThreads = 256;
constexpr int kColumnThreads = 128;

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

// Adds up the partials: 32 columns of dweight and dbias per block, sixteen warps each
// taking every sixteenth partial, in a fixed order. (part is not __restrict__: its loads stay
// behind the wait for the launch that writes it.)
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps)
    layer_norm_join_kernel(const float* part, int ranges, int D, void* dweight,
                           void* dbias, int wbf16) {
  __shared__ float2 s_sum[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float2 s = make_float2(0.f, 0.f);
  wait_for_launch_before();
  if (i < D) {
#pragma unroll 10
    for (int r = warp; r < ranges; r += kJoinWarps) {
      s.x += part[static_cast<int64_t>(r) * 2 * D + i];
      s.y += part[static_cast<int64_t>(r) * 2 * D + D + i];
    }
  }
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < D) {
#pragma unroll
    for (int q = 1; q < kJoinWarps; ++q) {
      s.x += s_sum[q][lane].x;
      s.y += s_sum[q][lane].y;
    }
    if (dweight != nullptr) store_from_f32(dweight, i, s.x, wbf16);
    if (dbias != nullptr) store_from_f32(dbias, i, s.y, wbf16);
  }
}

// ---- rows held in registers ---------------------------------------------------------

// Sum of a pair over the R threads of a group (R a multiple of 32, at most the block);
// the same value in all of them. `slots` are the block's warps' slots, not read by any
// warp that has not passed a block barrier since the call before last.
__device__ __forceinline__ float2 group_sum2(float2 v, int R, float2* slots) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (R == 32) return v;
  if (lane == 0) slots[warp] = v;
  __syncthreads();
  const int per = R >> 5, base = warp - warp % per;
  v = lane < per ? slots[base + lane] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

template <int kBf16, int VW, int kNv>
__global__ void __launch_bounds__(1024, kNv * (Pack<kBf16, VW>::kBytes + 3) / 4 <= 8 && VW > 1 ? 2 : 1)
    layer_norm_rows_kernel(const void* x, int64_t ldx, const void* weight, const void* bias,
                           int wbf16, int N, int D, float eps, void* y, int64_t ldy,
                           float* mean_out, float* rstd_out, int R) {
  using P = Pack<kBf16, VW>;
  __shared__ float2 s_slots[2][32];
  const int group = threadIdx.x / R, t = threadIdx.x % R;
  const int row = blockIdx.x * (blockDim.x / R) + group;
  const int nvec = row < N ? D / VW : 0;
  const int64_t xr = static_cast<int64_t>(row) * ldx, yr = static_cast<int64_t>(row) * ldy;
  typename P::Raw raw[kNv];   // as loaded: half the registers of widened bf16
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kNv; ++k)
    if (t + k * R < nvec) raw[k] = P::load(x, xr + static_cast<int64_t>(t + k * R) * VW);
#pragma unroll
  for (int k = 0; k < kNv; ++k)
    if (t + k * R < nvec) {
      float v[VW];
      P::widen(raw[k], v);
#pragma unroll
      for (int e = 0; e < VW; ++e) sum += v[e];
    }
  const float inv_d = 1.f / static_cast<float>(D);
  const float mean = group_sum2(make_float2(sum, 0.f), R, s_slots[0]).x * inv_d;
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < kNv; ++k)
    if (t + k * R < nvec) {
      float v[VW];
      P::widen(raw[k], v);
#pragma unroll
      for (int e = 0; e < VW; ++e) sq = fmaf(v[e] - mean, v[e] - mean, sq);
    }
  const float rstd = 1.f / sqrtf(group_sum2(make_float2(sq, 0.f), R, s_slots[1]).x * inv_d + eps);
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    const int i = t + k * R;
    if (i < nvec) {
      float v[VW], w[VW], b[VW];
      P::widen(raw[k], v);
      load_param<VW>(weight, i * VW, wbf16, 1.f, w);
      load_param<VW>(bias, i * VW, wbf16, 0.f, b);
#pragma unroll
      for (int e = 0; e < VW; ++e) v[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
      P::store(y, yr + static_cast<int64_t>(i) * VW, v);
    }
  }
  if (t == 0 && row < N) {
    if (mean_out != nullptr) mean_out[row] = mean;
    if (rstd_out != nullptr) rstd_out[row] = rstd;
  }
}

// dx and, in part (not null), this CTA's sums over its rows: part[blockIdx.x][0][i] of dy h
// and [1][i] of dy.
template <int kBf16, int VW, int kNv>
__global__ void __launch_bounds__(512, kNv * VW <= 8 && VW > 1 ? 2 : 1)
    layer_norm_grad_kernel(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                           const void* weight, int wbf16, const float* __restrict__ mean_in,
                           const float* __restrict__ rstd_in, int N, int D, void* dx,
                           int64_t lddx, float* part, int R) {
  using P = Pack<kBf16, VW>;
  using Raw = typename P::Raw;
  __shared__ float2 s_slots[2][16];
  extern __shared__ float s_cols[];   // [groups][2 * D] when several groups share a block
  start_next_launch();
  const int groups = blockDim.x / R;
  const int group = threadIdx.x / R, t = threadIdx.x % R;
  const int nvec = D / VW;
  const int step = gridDim.x * groups;
  const float inv_d = 1.f / static_cast<float>(D);
  float dw[kNv][VW], db[kNv][VW], w[kNv][VW];
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
#pragma unroll
    for (int e = 0; e < VW; ++e) dw[k][e] = db[k][e] = 0.f;
    if (t + k * R < nvec) load_param<VW>(weight, (t + k * R) * VW, wbf16, 1.f, w[k]);
  }
  Raw rx[kNv], rg[kNv];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int row) {
    if (row < N) {
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        const int i = t + k * R;
        if (i < nvec) {
          rx[k] = P::load(x, static_cast<int64_t>(row) * ldx + static_cast<int64_t>(i) * VW);
          rg[k] = P::load(dy, static_cast<int64_t>(row) * lddy + static_cast<int64_t>(i) * VW);
        }
      }
      mean = mean_in[row];
      rstd = rstd_in[row];
    }
  };
  int row = blockIdx.x * groups + group;
  fetch(row);
  // every group of the grid takes as many turns, for the block barriers of the sums
  const int turns = (N + step - 1) / step;
  for (int turn = 0; turn < turns; ++turn, row += step) {
    const bool live = row < N;
    const float r = rstd;
    float g[kNv][VW], h[kNv][VW];
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kNv; ++k)
      if (live && t + k * R < nvec) {
        P::widen(rx[k], h[k]);
        P::widen(rg[k], g[k]);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          h[k][e] = (h[k][e] - mean) * r;
          dw[k][e] = fmaf(g[k][e], h[k][e], dw[k][e]);
          db[k][e] += g[k][e];
          g[k][e] *= w[k][e];
          sum.x += g[k][e];
          sum.y = fmaf(g[k][e], h[k][e], sum.y);
        }
      }
    fetch(row + step);
    if (dx != nullptr) {
      sum = group_sum2(sum, R, s_slots[turn & 1]);
      const float mg = sum.x * inv_d, mgh = sum.y * inv_d;
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        const int i = t + k * R;
        if (live && i < nvec) {
#pragma unroll
          for (int e = 0; e < VW; ++e) g[k][e] = r * (g[k][e] - mg - h[k][e] * mgh);
          P::store(dx, static_cast<int64_t>(row) * lddx + static_cast<int64_t>(i) * VW, g[k]);
        }
      }
    }
  }
  if (part == nullptr) return;
  float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * D;
  if (groups > 1) out = s_cols + static_cast<int64_t>(group) * 2 * D;
#pragma unroll
  for (int k = 0; k < kNv; ++k) {
    const int i = t + k * R;
    if (i < nvec) {
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        out[i * VW + e] = dw[k][e];
        out[D + i * VW + e] = db[k][e];
      }
    }
  }
  if (groups > 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
      float s = 0.f;
      for (int q = 0; q < groups; ++q) s += s_cols[q * 2 * D + i];
      part[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = s;
    }
  }
}

}  // namespace

namespace {

// Threads per row: enough for nvec vectors at `most` per thread, and then more, down to
// one vector per thread, while the rows alone do not fill the GPU (a quarter of its 2048
// threads per SM).
int row_threads(int nvec, int most, int limit, int64_t N, int sms) {
  int R = 32;
  while (R * most < nvec) R *= 2;
  while (R < nvec && R < limit && N * R < static_cast<int64_t>(sms) * 512) R *= 2;
  return R;
}

// Vectors of a row that a thread of the forward kernel holds at most: 16 elements.
constexpr int norm_vectors(int vw) { return 16 / vw; }

template <int kBf16, int VW>
cudaError_t norm_rows(const void* x, int64_t ldx, const void* weight, const void* bias, int wbf16,
                      int N, int D, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                      int sms, cudaStream_t stream) {
  constexpr int kMost = norm_vectors(VW);
  const int nvec = D / VW;
  const int R = row_threads(nvec, kMost, 1024, N, sms);
  const int block = R < 128 ? 128 : R;
  const int rows = block / R;
  auto go = [&](auto kern) {
    kern<<<(N + rows - 1) / rows, block, 0, stream>>>(x, ldx, weight, bias, wbf16, N, D, eps, y,
                                                      ldy, mean, rstd, R);
    return cudaGetLastError();
  };
  const int per = (nvec + R - 1) / R;
  if (per <= 1) return go(layer_norm_rows_kernel<kBf16, VW, 1>);
  if (per <= 2) return go(layer_norm_rows_kernel<kBf16, VW, 2>);
  if constexpr (kMost >= 4)
    if (per <= 4) return go(layer_norm_rows_kernel<kBf16, VW, 4>);
  if constexpr (kMost >= 8)
    if (per <= 8) return go(layer_norm_rows_kernel<kBf16, VW, 8>);
  return go(layer_norm_rows_kernel<kBf16, VW, kMost>);
}

// The backward kernel: 512 threads per CTA, several rows at a time where a row needs fewer,
// each thread holding 8 elements of a row (two CTAs per SM by registers), or 16 for rows
// of more than 4096 (one CTA).
constexpr int kGradBlock = 512;
constexpr int grad_elems(int vw) { return vw == 1 ? 8 : 16; }

template <int kBf16, int VW>
cudaError_t norm_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight,
                      int wbf16, const float* mean, const float* rstd, int N, int D, void* dx,
                      int64_t lddx, float* part, int* ranges, int sms, cudaStream_t stream) {
  constexpr int kMost = grad_elems(VW) / VW;
  const int nvec = D / VW;
  const int R = row_threads(nvec, nvec <= kGradBlock * 8 / VW ? 8 / VW : kMost, kGradBlock, N, sms);
  const int groups = kGradBlock / R;
  const size_t smem = groups > 1 ? static_cast<size_t>(groups) * 2 * D * 4 : 0;   // at most 32 KB
  int grid = (N + groups - 1) / groups;
  if (grid > kNormRanges) grid = kNormRanges;
  *ranges = grid;
  auto go = [&](auto kern) {
    kern<<<grid, kGradBlock, smem, stream>>>(dy, lddy, x, ldx, weight, wbf16, mean, rstd, N, D,
                                             dx, lddx, part, R);
    return cudaGetLastError();
  };
  const int per = (nvec + R - 1) / R;
  if (per <= 1) return go(layer_norm_grad_kernel<kBf16, VW, 1>);
  if (per <= 2) return go(layer_norm_grad_kernel<kBf16, VW, 2>);
  if constexpr (kMost >= 4)
    if (per <= 4) return go(layer_norm_grad_kernel<kBf16, VW, 4>);
  return go(layer_norm_grad_kernel<kBf16, VW, kMost>);
}

cudaError_t join_columns(const float* part, int ranges, int D, void* dweight, void* dbias,
                         int wbf16, cudaStream_t stream) {
  return launch_after(layer_norm_join_kernel, dim3(static_cast<unsigned>((D + 31) / 32)),
                      dim3(32 * kJoinWarps), 0, stream, part, ranges, D, dweight, dbias, wbf16);
}

}  // namespace

cudaError_t launch_layer_norm(const void* x, int bf16, int64_t ldx, const void* weight,
                              const void* bias, int wbf16, int N, int D, float eps, void* y,
                              int64_t ldy, float* mean, float* rstd, int sms,
                              cudaStream_t stream) {
  if (norm_stream_fits(D, bf16 ? 2 : 4)) {
    const cudaError_t e = launch_norm_stream(x, bf16, ldx, weight, bias, wbf16, N, D, eps, y, ldy,
                                             mean, rstd, sms, stream);
    if (e != cudaErrorNotSupported) return e;   // few rows: the kernel below
  }
  const int vw = access_width(bf16, D, {ldx, ldy}, {x, y}, {weight, bias}, wbf16);
  if (D / vw <= 1024 * norm_vectors(vw)) {
    auto go = [&](auto f) {
      return f(x, ldx, weight, bias, wbf16, N, D, eps, y, ldy, mean, rstd, sms, stream);
    };
    if (bf16) {
      switch (vw) {
        case 8: return go(norm_rows<1, 8>);
        case 4: return go(norm_rows<1, 4>);
        case 2: return go(norm_rows<1, 2>);
        default: return go(norm_rows<1, 1>);
      }
    }
    switch (vw) {
      case 4: return go(norm_rows<0, 4>);
      case 2: return go(norm_rows<0, 2>);
      default: return go(norm_rows<0, 1>);
    }
  }
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
  const bool columns = dweight != nullptr || dbias != nullptr;
  int ranges = 0;
  if (N > 0 && norm_stream_fits(D, bf16 ? 2 : 4)) {
    e = launch_norm_stream_backward(dy, lddy, x, bf16, ldx, weight, wbf16, mean, rstd, N, D, dx,
                                    lddx, dweight, dbias, columns ? part : nullptr, &ranges, sms,
                                    stream);
    if (e == cudaSuccess && columns && ranges > 1)
      return join_columns(part, ranges, D, dweight, dbias, wbf16, stream);
    if (e != cudaErrorNotSupported) return e;
    e = cudaSuccess;
  }
  const int vw = access_width(bf16, D, {lddy, ldx, dx != nullptr ? lddx : 0}, {dy, x, dx}, {weight},
                              wbf16);
  if (N > 0 && D <= grad_elems(vw) * kGradBlock) {
    auto go = [&](auto f) {
      return f(dy, lddy, x, ldx, weight, wbf16, mean, rstd, N, D, dx, lddx,
               columns ? part : nullptr, &ranges, sms, stream);
    };
    if (bf16) {
      switch (vw) {
        case 8: e = go(norm_grad<1, 8>); break;
        case 4: e = go(norm_grad<1, 4>); break;
        case 2: e = go(norm_grad<1, 2>); break;
        default: e = go(norm_grad<1, 1>); break;
      }
    } else {
      switch (vw) {
        case 4: e = go(norm_grad<0, 4>); break;
        case 2: e = go(norm_grad<0, 2>); break;
        default: e = go(norm_grad<0, 1>); break;
      }
    }
  } else if (N > 0) {
    // the column sums first: dx may overwrite dy
    if (columns) {
      ranges = N < kNormRanges ? N : kNormRanges;
      const dim3 grid(static_cast<unsigned>((D + kColumnThreads - 1) / kColumnThreads),
                      static_cast<unsigned>(ranges));
      layer_norm_columns_kernel<<<grid, kColumnThreads, 0, stream>>>(dy, lddy, x, bf16, ldx, mean,
                                                                     rstd, N, D, ranges, part);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    if (dx != nullptr) {
      const int grid = N < sms * 8 ? N : sms * 8;
      layer_norm_dx_kernel<<<grid, kNormThreads, 0, stream>>>(dy, lddy, x, bf16, ldx, weight,
                                                              wbf16, mean, rstd, N, D, dx, lddx);
      e = cudaGetLastError();
    }
  }
  if (e != cudaSuccess || !columns) return e;
  return join_columns(part, ranges, D, dweight, dbias, wbf16, stream);
}

}  // namespace flce
