// Per-token work around the log-probability GEMMs: joining the vocabulary ranges'
// partial sums and rankings into the outputs, and the gradient's row coefficients. A few
// microseconds beside products of 190 us and more.
#include <cstdint>

#include "flce_internal.h"
#include "flce_rowstat.cuh"
#include "flce_topk.cuh"

namespace flce {

namespace {

constexpr int kMergeWarps = 8;

// One warp per token (kWide = 0), or, with many ranges (few tokens), a block of eight
// warps per token, each joining every eighth range.
template <int kWide>
__global__ void __launch_bounds__(32 * kMergeWarps)
    logprob_merge_kernel(const float4* __restrict__ part, const float* __restrict__ zt,
                         const uint64_t* __restrict__ lists, const int32_t* __restrict__ tokens,
                         int N, int V, int part_stride, int splits, int ignore_index, int top_k,
                         float inv_t, float* __restrict__ logprob, float* __restrict__ entropy,
                         float* __restrict__ lse, float* __restrict__ top_lp,
                         int32_t* __restrict__ top_id, int32_t* status) {
  __shared__ float s_part[kMergeWarps][3];
  __shared__ uint64_t s_list[kMergeWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = kWide ? blockIdx.x : blockIdx.x * kMergeWarps + warp;
  if (!kWide && i >= N) return;
  const float c = kLog2e * inv_t;
  const int first = kWide ? warp : 0;
  constexpr int kStep = kWide ? kMergeWarps : 1;
  auto slot = [&](int s) { return static_cast<int64_t>(s) * part_stride * BM + i; };

  RowPart p{-INFINITY, 0.f, 0.f};
  for (int s = first + lane * kStep; s < splits; s += 32 * kStep) {
    const float4 q = part[slot(s)];
    row_join(p, RowPart{q.x, q.y, q.z}, c);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const RowPart q{__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.s, o),
                    __shfl_xor_sync(0xffffffffu, p.t, o)};
    row_join(p, q, c);
  }
  uint64_t list = 0;
  if (top_k > 0) {
    // 32 keys at a time, of as many ranges as they are
    for (int b = first * 32; b < splits * top_k; b += 32 * kStep) {
      const int s = (b + lane) / top_k, j = b + lane - s * top_k;
      const uint64_t k = warp_sort_desc(s < splits ? lists[slot(s) * top_k + j] : 0, lane);
      list = b == first * 32 ? k : warp_merge_desc(list, k, lane);
    }
  }
  if (kWide) {
    if (lane == 0) {
      s_part[warp][0] = p.m;
      s_part[warp][1] = p.s;
      s_part[warp][2] = p.t;
    }
    s_list[warp][lane] = list;
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < kMergeWarps; ++w) {
      row_join(p, RowPart{s_part[w][0], s_part[w][1], s_part[w][2]}, c);
      if (top_k > 0) list = warp_merge_desc(list, s_list[w][lane], lane);
    }
  }
  const int y = tokens != nullptr ? tokens[i] : ignore_index;
  const bool bad = y != ignore_index && (y < 0 || y >= V);
  const bool has = y != ignore_index && !bad;
  const RowOut r = row_finish(p, has ? zt[i] : 0.f, has, inv_t, c);
  if (lane == 0) {
    if (logprob != nullptr) logprob[i] = bad ? __uint_as_float(0x7FC00000u) : r.logprob;
    if (entropy != nullptr) entropy[i] = r.entropy;
    if (lse != nullptr) lse[i] = r.lse;
    if (bad && status != nullptr) atomicCAS(reinterpret_cast<int*>(status), 0, 8);
  }
  if (lane < top_k) {
    const int64_t at = static_cast<int64_t>(i) * top_k + lane;
    top_id[at] = list == 0 ? -1 : key_id(list);
    top_lp[at] = r.lse != r.lse ? r.lse
                 : list == 0    ? -INFINITY
                                : id_logprob(r, key_value(list), inv_t);
  }
}

__global__ void logprob_coef_kernel(const int32_t* __restrict__ tokens, int N, int V,
                                    int ignore_index, float inv_t,
                                    const float* __restrict__ logprob,
                                    const float* __restrict__ entropy,
                                    const float* __restrict__ lse,
                                    const float* __restrict__ dlogprob,
                                    const float* __restrict__ dentropy,
                                    const float* __restrict__ dlse, float4* __restrict__ coef,
                                    float* __restrict__ target) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= N) return;
  const int y = tokens != nullptr ? tokens[i] : ignore_index;
  const bool has = y != ignore_index && y >= 0 && y < V;
  const RowCoef k = row_coef(lse[i], entropy != nullptr ? entropy[i] : 0.f,
                             logprob != nullptr ? logprob[i] : 0.f,
                             dlogprob != nullptr ? dlogprob[i] : 0.f,
                             dentropy != nullptr ? dentropy[i] : 0.f,
                             dlse != nullptr ? dlse[i] : 0.f, has, inv_t);
  coef[i] = make_float4(k.lse, k.A, k.B, k.entropy);
  target[i] = k.target;
}

}  // namespace

cudaError_t launch_logprob_merge(const float4* part, const float* zt, const uint64_t* lists,
                                 const int32_t* tokens, int N, int V, int part_stride, int splits,
                                 int ignore_index, int top_k, float inv_t, float* logprob,
                                 float* entropy, float* lse, float* top_lp, int32_t* top_id,
                                 int32_t* status, cudaStream_t stream) {
  auto go = [&](auto kern, int grid) {
    kern<<<grid, 32 * kMergeWarps, 0, stream>>>(part, zt, lists, tokens, N, V, part_stride, splits,
                                                ignore_index, top_k, inv_t, logprob, entropy, lse,
                                                top_lp, top_id, status);
    return cudaGetLastError();
  };
  // Many ranges come with few tokens. D = 4096, V = 128256, 20 alternatives, the call with a block
  // / a warp per token: 129 tokens (76 ranges) 210 / 241 us, 768 (25) 538 / 571, 2048 (9) 1277 / 1259.
  return splits > 2 * kMergeWarps
             ? go(logprob_merge_kernel<1>, N)
             : go(logprob_merge_kernel<0>, (N + kMergeWarps - 1) / kMergeWarps);
}

cudaError_t launch_logprob_coef(const int32_t* tokens, int N, int V, int ignore_index, float inv_t,
                                const float* logprob, const float* entropy, const float* lse,
                                const float* dlogprob, const float* dentropy, const float* dlse,
                                float4* coef, float* target, cudaStream_t stream) {
  logprob_coef_kernel<<<(N + 255) / 256, 256, 0, stream>>>(tokens, N, V, ignore_index, inv_t,
                                                           logprob, entropy, lse, dlogprob,
                                                           dentropy, dlse, coef, target);
  return cudaGetLastError();
}

}  // namespace flce
