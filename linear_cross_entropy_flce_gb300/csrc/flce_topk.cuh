// Ranking keys and warp-wide sorted lists for the most likely ids of a row.
//
// A key is 64 bits: the logit, mapped to an unsigned integer of the same order, above
// the complement of its id. Larger key = larger logit, and among equal logits the
// lower id, so one unsigned comparison ranks (value, id) pairs and any order of
// merging gives the same list. Key 0 is an empty slot (below every real key).
//
// A warp holds a list of up to 32 keys, one per lane, in descending order. Two sorted
// lists merge to the 32 largest of both in six steps: the element-wise maximum of one
// with the other reversed holds them as a bitonic sequence, which five compare-exchange
// steps sort.
#pragma once

#include <cmath>
#include <cstdint>

namespace flce {

constexpr int kMaxTopK = 32;

// Bits that order as the values do.
__device__ __forceinline__ uint32_t ordered_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);   // -0 ranks as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

__device__ __forceinline__ uint64_t rank_key(float v, int id) {
  return (static_cast<uint64_t>(ordered_bits(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

__device__ __forceinline__ float key_value(uint64_t k) {
  return ordered_value(static_cast<uint32_t>(k >> 32));
}

__device__ __forceinline__ int key_id(uint64_t k) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
}

// Compare-exchange with the lane `mask` away: the lane keeps the larger key if
// `keep_max`.
__device__ __forceinline__ uint64_t key_exchange(uint64_t k, int mask, bool keep_max) {
  const uint64_t o = __shfl_xor_sync(0xffffffffu, k, mask);
  return (k > o) == keep_max ? k : o;
}

// Bitonic sequence over the warp to descending order.
__device__ __forceinline__ uint64_t warp_bitonic_desc(uint64_t k, int lane) {
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) k = key_exchange(k, j, (lane & j) == 0);
  return k;
}

// Any 32 keys to descending order.
__device__ __forceinline__ uint64_t warp_sort_desc(uint64_t k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
    const bool desc = (lane & size) == 0 || size == 32;
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1) k = key_exchange(k, j, ((lane & j) == 0) == desc);
  }
  return k;
}

// The 32 largest of two descending lists, in descending order.
__device__ __forceinline__ uint64_t warp_merge_desc(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
  return warp_bitonic_desc(a > r ? a : r, lane);
}

}  // namespace flce
