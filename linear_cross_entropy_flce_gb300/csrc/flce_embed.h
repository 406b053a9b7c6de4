// Embedding lookup and its gradient (flce_embed.cu, flce_embed_sort.cu).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace flce {

// Tokens that are sorted by counting. In us of a whole gradient onto a table of 64, by passes / by counting: 64
// tokens 10.4 / 6.5, 1000 13.6 / 8.0, 4000 23.7 / 20.5, 8192 25.8 / 29.5.
constexpr int kSortCount = 4096;
// Tokens that one cluster sorts, in shared memory; more are sorted in tiles.
constexpr int kSortCluster = 16384;
constexpr int kSortTile = 4096;
constexpr int kSortDigitBits = 9;

// Positions of the sorted order that one CTA adds up: few for few tokens, so that they are spread over the
// GPU, else 32 (more partial rows cost more than they give), and more where that would make more than 2048
// ranges, whose partial rows the workspace holds. In us with 8 / 16 / 32, onto a table of 4096 bf16: 1000 tokens
// 11.8 / 13.2 / 15.8, 2000 17.7 / 17.1 / 19.1, 4000 28.5 / 24.4 / 23.9, 8192 53.7 / 45.9 / 41.3; of 1111 fp32 2000
// 15.8 / 15.4 / 19.1.
inline int embed_range(int64_t N) {
  if (N <= 1024) return 8;
  if (N <= 2048) return 16;
  const int64_t t = (N + 2047) / 2048;
  return static_cast<int>(std::max<int64_t>(32, (t + 7) / 8 * 8));
}

struct EmbedPlan {
  int64_t ranges, tiles;
  size_t off_ids, off_perm, off_ids2, off_perm2, off_counts, off_part, total;
};

inline EmbedPlan make_embed_plan(int64_t N, int64_t D) {
  EmbedPlan p;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  p.ranges = (N + embed_range(N) - 1) / embed_range(N);
  p.tiles = N <= kSortCluster ? 0 : (N + kSortTile - 1) / kSortTile;
  const size_t n4 = static_cast<size_t>(N) * 4;
  p.off_ids = take(n4);
  p.off_perm = take(n4);
  p.off_ids2 = take(p.tiles > 0 ? n4 : 0);
  p.off_perm2 = take(p.tiles > 0 ? n4 : 0);
  p.off_counts = take(p.tiles > 0 ? (static_cast<size_t>(p.tiles) << kSortDigitBits) * 4 : 0);
  p.off_part = take(static_cast<size_t>(p.ranges) * 2 * static_cast<size_t>(D) * 4);
  p.total = at;
  return p;
}

// ids[i], perm[i]: the tokens sorted by id, stably, and where they were; ids outside [0, V),
// ignore_index among them, come last as V. (ids2, perm2, counts: scratch for several tiles.)
cudaError_t launch_sort_tokens(const int32_t* tokens, int N, int V, int ignore_index, uint32_t* ids,
                               uint32_t* perm, uint32_t* ids2, uint32_t* perm2, uint32_t* counts,
                               cudaStream_t stream);

cudaError_t launch_embedding(const void* weight, int wbf16, int64_t ldw, const int32_t* tokens,
                             int N, int V, int D, float scale, int ignore_index, void* y, int bf16,
                             int64_t ldy, int32_t* status, cudaStream_t stream);

cudaError_t launch_embedding_grad(const void* dy, int bf16, int64_t lddy, const uint32_t* ids,
                                  const uint32_t* perm, int N, int V, int D, float scale, void* dW,
                                  int wbf16, int64_t ldw, int accumulate, float* part,
                                  cudaStream_t stream);

}  // namespace flce
