// The ring through which the streaming layer-norm kernels read their rows.
//
// A CTA has groups of R threads, each of which walks its own rows (first, first + step, ...)
// through a ring of kRing turns' rows in shared memory, filled by the bulk-copy engine: one thread
// starts a row's copy, nobody spends registers or instructions on loads in flight, and 100 KB
// or more per SM are on their way at any time. The engine copies 16-byte chunks, so that the
// rows, their stride and their length have to be multiples of 16 bytes; other rows are read
// element by element anyway, and the kernels of flce_norm.cu do that faster from registers.
#pragma once

#include <cstdint>

#include "flce_norm.cuh"
#include "ptx.cuh"

namespace flce {
namespace {

constexpr int kStreamVectors = 4;    // 16-byte vectors of a row per thread at most
constexpr uint64_t kStreamWaitNs = 2000000000ull;

// Barrier of the R threads of a group.
__device__ __forceinline__ void group_sync(int group, int R) {
  if (R == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(R) : "memory");
}

// Sum over the group, the same in all of its threads; one barrier. `slots` (a float2 per warp
// of the CTA) must not be written again before another barrier of the group.
__device__ __forceinline__ float2 stream_sum2(float2 v, int group, int R, float2* slots) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (R == 32) return v;
  if (lane == 0) slots[warp] = v;
  group_sync(group, R);
  const int per = R >> 5, base = group * per;
  float2 s = slots[base];
#pragma unroll 4
  for (int w = 1; w < per; ++w) {
    const float2 o = slots[base + w];
    s.x += o.x;
    s.y += o.y;
  }
  return s;
}
// one thread: starts the copy of a row of `bytes` (a multiple of 16, both sides aligned)
__device__ __forceinline__ void ring_copy(uint32_t slot, const void* row, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(slot),
      "l"(row), "r"(bytes), "r"(bar)
      : "memory");
}

// Threads per row, a multiple of 32, and groups per CTA of at most `block` threads whose
// rings (`ring_bytes` each) fit beside `fixed` bytes; 0 groups if none does.
struct StreamShape {
  int R, groups;
  size_t smem;
};
inline StreamShape stream_shape(int nvec, int64_t turns, int block, size_t ring_bytes, size_t fixed,
                                int sms) {
  StreamShape s;
  s.R = ((nvec + kStreamVectors - 1) / kStreamVectors + 31) / 32 * 32;
  s.groups = block / s.R;
  constexpr size_t kMost = 224 * 1024;
  while (s.groups > 0 && fixed + s.groups * ring_bytes > kMost) --s.groups;
  const int64_t per_sm = (turns + sms - 1) / sms;   // few rows: spread over the SMs
  if (s.groups > per_sm) s.groups = static_cast<int>(per_sm);
  s.smem = fixed + static_cast<size_t>(s.groups) * ring_bytes;
  return s;
}

// f(vectors per thread): all but the last are inside the row for every thread.
template <typename F>
cudaError_t with_stream_vectors(int per, F&& f) {
  static_assert(kStreamVectors == 4, "the cases below");
  if (per <= 2) return f(std::integral_constant<int, 2>{});
  if (per == 3) return f(std::integral_constant<int, 3>{});
  return f(std::integral_constant<int, 4>{});
}

// f(bf16, wbf16) with the values as compile-time constants.
template <typename F>
cudaError_t with_stream_types(int bf16, int wbf16, F&& f) {
  using One = std::integral_constant<int, 1>;
  using Zero = std::integral_constant<int, 0>;
  if (bf16) return wbf16 ? f(One{}, One{}) : f(One{}, Zero{});
  return wbf16 ? f(Zero{}, One{}) : f(Zero{}, Zero{});
}

}  // namespace
}  // namespace flce
