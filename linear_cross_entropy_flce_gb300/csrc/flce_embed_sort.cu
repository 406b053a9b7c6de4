// Tokens sorted by id, stably: radix passes of up to 9 bits.
//
// A CTA ranks a tile of items by a digit. Its 32 warps own consecutive parts of the tile and
// walk them 32 items at a time: lanes with equal digits find one another with match.any, and the
// first of them advances the warp's counter of that digit, so that an item's rank among its
// warp's equals is known and order is kept. Then the counters of all warps are summed digit by
// digit, and every item knows its place.
//
// Up to 16384 tokens one cluster of 8 CTAs takes all passes: each has a consecutive part of the items, reads
// the others' digit counts and puts every item where it goes, in the shared memory of whichever CTA owns
// that place. More tokens go through tiles with three launches a pass (count, offsets of every digit and
// tile, place). Up to kSortCount tokens, finally, are counted against one another without any passes.
//
// Bound by latency: barriers and dependent accesses to shared memory. 8192 tokens of 128256 ids, two passes, 11 us
// (23 by one CTA with eight items a thread), 65536 of 32000 35 in six launches.
#include <cstdint>

#include "flce_embed.h"
#include "flce_launch.cuh"
#include "ptx.cuh"

namespace flce {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1 << kSortDigitBits;

struct SortShared {
  uint16_t count[kWarps][kBins];   // a tile has at most 4096 items
  uint32_t total[kBins];           // of the tile
  uint32_t base[kBins];
  uint32_t warp_sum[kWarps];
};

__device__ __forceinline__ uint32_t key_of(const int32_t* tokens, int i, int V, int ignore_index) {
  const int32_t t = tokens[i];
  return t == ignore_index || t < 0 || t >= V ? static_cast<uint32_t>(V) : static_cast<uint32_t>(t);
}

// Item j of this thread is at warp * 32 * kItems + j * 32 + lane.
template <int kItems>
__device__ __forceinline__ int item_at(int j) {
  return (threadIdx.x >> 5) * 32 * kItems + j * 32 + (threadIdx.x & 31);
}

// place[j]: for each of this thread's items (n of them in the tile, keys in key) its rank by the digit at
// `shift` among the equal ones of its warp; sh.count: the equal ones in the warps before; sh.total: all of the
// tile's. Ends with a barrier.
template <int kItems>
__device__ __forceinline__ void rank_tile(SortShared& sh, const uint32_t (&key)[kItems], int n, int shift,
                                          int bits, uint32_t (&place)[kItems]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t mask = (1u << bits) - 1u;
  const int bins = 1 << bits;
  const int warps = min(kWarps, (n + 32 * kItems - 1) / (32 * kItems));   // that have items
  if (warp < warps)
    for (int b = lane; b < bins / 2; b += 32) reinterpret_cast<uint32_t*>(sh.count[warp])[b] = 0;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    if (warp >= warps) break;
    const bool in = item_at<kItems>(j) < n;
    const uint32_t d = in ? (key[j] >> shift) & mask : kBins;   // kBins: no item
    const uint32_t peers = __match_any_sync(0xffffffffu, d);
    const int first = __ffs(static_cast<int>(peers)) - 1;
    uint32_t before = 0;
    if (in && lane == first) {
      before = sh.count[warp][d];
      sh.count[warp][d] = static_cast<uint16_t>(before + __popc(peers));
    }
    before = __shfl_sync(0xffffffffu, before, first);
    place[j] = before + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
  }
  __syncthreads();
  if (threadIdx.x < bins) {
    uint32_t total = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const uint32_t c = sh.count[w][threadIdx.x];
      sh.count[w][threadIdx.x] = static_cast<uint16_t>(total);
      total += c;
    }
    sh.total[threadIdx.x] = total;
  }
  __syncthreads();
}

// Of one value per thread, those of the threads before; two barriers.
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* warp_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  uint32_t all = lane < kWarps ? warp_sum[lane] : 0;   // each warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += up;
  }
  const uint32_t before = __shfl_sync(0xffffffffu, all, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return (warp > 0 ? before : 0) + sum - v;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_v2(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

constexpr int kCluster = 8;

// One cluster; CTA c has items [c per, (c + 1) per), per = 1024 kItems at most.
template <int kItems>
__global__ void __launch_bounds__(kThreads, 1)
    sort_cluster_kernel(const int32_t* tokens, int N, int V, int ignore_index, int bits, int passes, int per,
                        uint32_t* ids, uint32_t* perm) {
  __shared__ SortShared sh;
  extern __shared__ uint2 s_items[];   // [1024 kItems]: key, index
  start_next_launch();
  constexpr int ctas = kCluster;
  const int rank = static_cast<int>(cluster_ctarank());
  const int first = rank * per;
  const int n = N - first < per ? N - first : per;
  uint32_t key[kItems], index[kItems], place[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int i = item_at<kItems>(j);
    index[j] = static_cast<uint32_t>(first + i);
    key[j] = i < n ? key_of(tokens, first + i, V, ignore_index) : 0;
  }
  const int digit = (bits + passes - 1) / passes;
  for (int p = 0; p < passes; ++p) {
    const int shift = p * digit;
    const uint32_t mask = (1u << digit) - 1u;
    rank_tile<kItems>(sh, key, n, shift, digit, place);
    cluster_sync();   // every CTA's totals are there, and its items of the pass before are read
    // where this CTA's items of each digit begin: behind all smaller digits, and the CTAs before
    uint32_t all = 0, before = 0;
    if (threadIdx.x <= mask) {
      const uint32_t at = smem_u32(&sh.total[threadIdx.x]);
#pragma unroll
      for (int c = 0; c < ctas; ++c) {
        const uint32_t t = ld_cluster_u32(mapa_shared(at, static_cast<uint32_t>(c)));
        all += t;
        before += c < rank ? t : 0;
      }
    }
    const uint32_t smaller = sum_before(all, sh.warp_sum);
    if (threadIdx.x <= mask) sh.base[threadIdx.x] = smaller + before;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kItems; ++j)
      if (item_at<kItems>(j) < n) {
        const uint32_t d = (key[j] >> shift) & mask;
        place[j] += sh.base[d] + sh.count[threadIdx.x >> 5][d];
        if (p == passes - 1) {
          ids[place[j]] = key[j];
          perm[place[j]] = index[j];
        } else {
          const uint32_t owner = place[j] / static_cast<uint32_t>(per);
          st_cluster_v2(mapa_shared(smem_u32(&s_items[place[j] - owner * per]), owner), key[j], index[j]);
        }
      }
    // (also before the CTA leaves: the others read its totals)
    cluster_sync();
    if (p == passes - 1) break;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int i = item_at<kItems>(j);
      if (i < n) {
        const uint2 v = s_items[i];
        key[j] = v.x;
        index[j] = v.y;
      }
    }
  }
}

// ---- few tokens ----------------------------------------------------------------------

// A token's place is the number of tokens that come before it: a CTA counts for 32 of them, a lane each, its
// warps taking shares of all the keys, four at a time. N^2 comparisons, but no pass waits for another.
constexpr int kCountThreads = 256;
constexpr int kCountWarps = kCountThreads / 32;
__global__ void __launch_bounds__(kCountThreads)
    sort_count_all_kernel(const int32_t* tokens, int N, int V, int ignore_index, uint32_t* ids, uint32_t* perm) {
  extern __shared__ uint4 s_keys[];   // four keys each, past N the largest
  __shared__ uint32_t s_place[kCountWarps][32];
  start_next_launch();
  const int lane = threadIdx.x & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  const int vectors = (N + 3) / 4;
  uint32_t* const keys = reinterpret_cast<uint32_t*>(s_keys);
#pragma unroll 8
  for (int i = threadIdx.x; i < vectors * 4; i += kCountThreads)
    keys[i] = i < N ? key_of(tokens, i, V, ignore_index) : 0xFFFFFFFFu;
  __syncthreads();
  const int first = static_cast<int>(blockIdx.x) * 32, i = first + lane;
  const uint32_t key = i < N ? keys[i] : 0xFFFFFFFEu;
  uint32_t place = 0;
  const int share = (vectors + kCountWarps - 1) / kCountWarps;
  const int end = min(vectors, (warp + 1) * share);
  // of equal ids those before this CTA's tokens come first, those after it later
  auto count = [&](int from, int to, uint32_t below) {
#pragma unroll 4
    for (int j = from; j < to; ++j) {
      const uint4 k = s_keys[j];
      place += (k.x < below) + (k.y < below) + (k.z < below) + (k.w < below);
    }
  };
  const int begin = warp * share, own = first / 4;
  count(begin, min(end, own), key + 1u);
  count(max(begin, own), end, key);
  s_place[warp][lane] = place;
  __syncthreads();
  if (warp != 0) return;
  const uint32_t equal = __match_any_sync(0xffffffffu, key);   // and of this CTA's own the earlier ones
  place = __popc(equal & ((1u << lane) - 1u));
#pragma unroll
  for (int w = 0; w < kCountWarps; ++w) place += s_place[w][lane];
  if (i < N) {
    ids[place] = key;
    perm[place] = static_cast<uint32_t>(i);
  }
}

// ---- several tiles -------------------------------------------------------------------

constexpr int kTileItems = kSortTile / kThreads;
static_assert(kTileItems <= 4, "the counters hold 16 bits");

// keys null: the first pass, from the tokens
__global__ void __launch_bounds__(kThreads)
    sort_count_kernel(const int32_t* tokens, const uint32_t* keys, int N, int V, int ignore_index,
                      int shift, int bits, uint32_t* counts) {
  __shared__ uint32_t s_count[kBins];
  const int bins = 1 << bits;
  for (int b = threadIdx.x; b < bins; b += kThreads) s_count[b] = 0;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSortTile;
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const int64_t i = first + j * kThreads + threadIdx.x;
    if (i < N) {
      const uint32_t k = keys != nullptr ? keys[i] : key_of(tokens, static_cast<int>(i), V, ignore_index);
      atomicAdd(&s_count[(k >> shift) & (bins - 1u)], 1u);
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kThreads)
    counts[static_cast<int64_t>(b) * gridDim.x + blockIdx.x] = s_count[b];
}

// In place: the sum of the entries before each, one CTA.
__global__ void __launch_bounds__(kThreads) sort_offsets_kernel(uint32_t* counts, int64_t entries) {
  __shared__ uint32_t s_sum[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t carry = 0;
  for (int64_t at = 0; at < entries; at += kThreads * 4) {
    const int64_t i = at + threadIdx.x * 4;
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = i + k < entries ? counts[i + k] : 0;
    uint32_t sum = c[0] + c[1] + c[2] + c[3];
    const uint32_t own = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    uint32_t before = carry, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    before += sum - own;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k < entries) counts[i + k] = before;
      before += c[k];
    }
    carry += all;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    sort_place_kernel(const int32_t* tokens, const uint32_t* keys, const uint32_t* places, int N, int V,
                      int ignore_index, int shift, int bits, const uint32_t* offsets, uint32_t* ids,
                      uint32_t* perm) {
  __shared__ SortShared sh;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSortTile;
  const int n = static_cast<int>(N - first < kSortTile ? N - first : kSortTile);
  uint32_t key[kTileItems], place[kTileItems];
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const int i = item_at<kTileItems>(j);
    key[j] = i >= n ? 0
             : keys != nullptr ? keys[first + i]
                               : key_of(tokens, static_cast<int>(first + i), V, ignore_index);
  }
  const int bins = 1 << bits;
  for (int b = threadIdx.x; b < bins; b += kThreads)
    sh.base[b] = offsets[static_cast<int64_t>(b) * gridDim.x + blockIdx.x];
  rank_tile<kTileItems>(sh, key, n, shift, bits, place);
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    const int i = item_at<kTileItems>(j);
    if (i < n) {
      const uint32_t d = (key[j] >> shift) & (bins - 1u);
      place[j] += sh.base[d] + sh.count[threadIdx.x >> 5][d];
      ids[place[j]] = key[j];
      perm[place[j]] = places != nullptr ? places[first + i] : static_cast<uint32_t>(first + i);
    }
  }
}

}  // namespace

cudaError_t launch_sort_tokens(const int32_t* tokens, int N, int V, int ignore_index, uint32_t* ids,
                               uint32_t* perm, uint32_t* ids2, uint32_t* perm2, uint32_t* counts,
                               cudaStream_t stream) {
  int bits = 1;   // of the keys 0 to V
  while ((static_cast<int64_t>(V) >> bits) != 0) ++bits;
  const int passes = (bits + kSortDigitBits - 1) / kSortDigitBits;
  if (N <= kSortCount) {
    const int smem = (N + 3) / 4 * 16;   // 16 KB at most
    sort_count_all_kernel<<<(N + 31) / 32, kCountThreads, smem, stream>>>(tokens, N, V, ignore_index, ids, perm);
    return cudaGetLastError();
  }
  if (N <= kSortCluster) {
    constexpr int ctas = kCluster;
    const int per = ((N + ctas - 1) / ctas + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto go = [&](auto kern, int items) {
      cfg.dynamicSmemBytes = static_cast<size_t>(kThreads) * items * sizeof(uint2);
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(cfg.dynamicSmemBytes));
      if (e != cudaSuccess) return e;
      return cudaLaunchKernelEx(&cfg, kern, tokens, N, V, ignore_index, bits, passes, per, ids, perm);
    };
    return per <= kThreads ? go(sort_cluster_kernel<1>, 1) : go(sort_cluster_kernel<2>, 2);
  }
  const int tiles = (N + kSortTile - 1) / kSortTile;
  const int per = (bits + passes - 1) / passes;
  const uint32_t *keys = nullptr, *places = nullptr;
  for (int p = 0; p < passes; ++p) {
    // the last pass ends in ids and perm
    const bool second = (passes - 1 - p) % 2 != 0;
    uint32_t* const to_ids = second ? ids2 : ids;
    uint32_t* const to_perm = second ? perm2 : perm;
    sort_count_kernel<<<tiles, kThreads, 0, stream>>>(tokens, keys, N, V, ignore_index, p * per, per, counts);
    sort_offsets_kernel<<<1, kThreads, 0, stream>>>(counts, static_cast<int64_t>(tiles) << per);
    sort_place_kernel<<<tiles, kThreads, 0, stream>>>(tokens, keys, places, N, V, ignore_index, p * per, per,
                                                      counts, to_ids, to_perm);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    keys = to_ids;
    places = to_perm;
  }
  return cudaSuccess;
}

}  // namespace flce
