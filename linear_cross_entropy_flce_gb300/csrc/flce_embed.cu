// Embedding lookup and its gradient.
//
//   y_n = scale W[t_n],   dW_v = scale sum_{n: t_n = v} dy_n
//
// Lookup: threads side by side take vectors of a row, several at a time with their loads first.
//
// Gradient: with the tokens sorted by id (flce_embed_sort.cu), the sorted order is cut into
// equal ranges, whatever ids they hold, so that a frequent id is shared out and a rare one costs
// no more than its rows. A CTA adds up a range's rows of dy in fp32, kAhead rows' loads at a time, for
// 128 vectors of columns; at the end of an id it writes that row of dW, and where an id goes on beyond
// the range's ends the partial sum goes to the workspace, of two rows per range. A last launch
// joins those, in the order of the ranges. The rows of ids without tokens are zeroed by further
// CTAs of the first launch, which look the ids up in the sorted order.
//
// Bound by the bytes of dW for a large table, by dy for a small one: 8192 tokens x 4096 bf16 take 13.6 us
// looked up, 171 for the gradient of 128256 rows (0.97 of the copy rate) and 42 added to a table that is there
// (3600 rows; the sort 11, the ranges 25, the join 9, which overlap a little); 3001 x 1111 fp32 of 32000 rows
// 5.5 and 40; one token 1.9 us and, added to a table, 3.1. Ranges of 32: 8 make four times the partial rows, and 8 are what few tokens get.
#include <cstdint>

#include "flce_embed.h"
#include "flce_gemm_params.h"
#include "flce_launch.cuh"
#include "flce_norm.cuh"

namespace flce {

namespace {

// ---- lookup --------------------------------------------------------------------------

constexpr int kLookupThreads = 128;
// Vectors of a row per thread. One element at a time, 12 is best on the whole: over rows of 601 to 8191 elements, 64
// to 16384 tokens and three pairs of types (75 sizes) 8 takes 7 % longer and 16 3 %, which is ahead for long rows
// alone. In us with 8 / 12 / 16, bf16: 8192 x 601 9.8 / 8.0 / 8.8, 16384 x 2731 50 / 45 / 51, 8192 x 4001 36 / 34 / 31,
// 3001 x 8191 27 / 26 / 24; the bytes of 8192 x 4001 are 20: 2 bytes an access.
constexpr int lookup_vectors(int vw) { return vw == 1 ? 12 : 4; }

// X threads per row; VW elements at a time.
template <int kWbf16, int kBf16, int VW>
__global__ void __launch_bounds__(kLookupThreads)
    embedding_kernel(const void* weight, int64_t ldw, const int32_t* tokens, int N, int V, int nvec,
                     float scale, int ignore_index, void* y, int64_t ldy, int32_t* status, int X) {
  using In = Param<kWbf16, VW>;
  using Out = Param<kBf16, VW>;
  constexpr int kLookup = lookup_vectors(VW);
  const int row = blockIdx.x * (kLookupThreads / X) + static_cast<int>(threadIdx.x) / X;
  if (row >= N) return;
  const int t = static_cast<int>(threadIdx.x) % X;
  const int token = tokens[row];
  const bool live = token >= 0 && token < V && token != ignore_index;
  const float none = token == ignore_index ? 0.f : __uint_as_float(0x7FC00000u);
  const int first = static_cast<int>(blockIdx.y) * X * kLookup + t;
  if (!live && token != ignore_index && status != nullptr && first == 0)
    atomicCAS(reinterpret_cast<int*>(status), 0, kStatusLabelRange);
  const uint8_t* const from =
      static_cast<const uint8_t*>(weight) + (live ? token : 0) * ldw * (kWbf16 ? 2 : 4);
  uint8_t* const to = static_cast<uint8_t*>(y) + row * ldy * (kBf16 ? 2 : 4);
  In in[kLookup];
#pragma unroll
  for (int k = 0; k < kLookup; ++k)
    if (live && first + k * X < nvec) in[k].load(from, (first + k * X) * VW, 0.f);
#pragma unroll
  for (int k = 0; k < kLookup; ++k)
    if (first + k * X < nvec) {
      float v[VW];
      if (live) in[k].widen(v);
#pragma unroll
      for (int e = 0; e < VW; ++e) v[e] = live ? v[e] * scale : none;
      Out out;
      out.narrow(v);
      out.save(to, (first + k * X) * VW);
    }
}

// ---- gradient ------------------------------------------------------------------------

constexpr int kGradThreads = 128;
constexpr int kAhead = 8;
constexpr int kZeroRows = 32;      // rows of dW that one CTA looks up and zeroes

// The first sorted position whose id is at least v.
__device__ __forceinline__ int lower_bound(const uint32_t* ids, int N, uint32_t v) {
  int lo = 0, hi = N;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (ids[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// `sum` scaled, and (kAdd) added to old values.
template <int n, int kAdd>
__device__ __forceinline__ void finish_sum(float (&sum)[n], float scale, const float (&old)[n]) {
#pragma unroll
  for (int e = 0; e < n; ++e) sum[e] = kAdd ? fmaf(sum[e], scale, old[e]) : sum[e] * scale;
}

// What a thread has of a row: a vector of VW elements; where that is one element, four of them, kGradThreads
// apart, so that a CTA's piece of a row is not too short.
constexpr int row_parts(int vw) { return vw == 1 ? 4 : 1; }
template <int kBf16, int VW>
struct RowPart {
  static constexpr int kParts = row_parts(VW), kValues = kParts * VW;
  Param<kBf16, VW> p[kParts];
  // (what is behind the row stays unset, and is not saved)
  __device__ void load(const void* row, int i, int nvec) {
#pragma unroll
    for (int c = 0; c < kParts; ++c)
      if (i + c * kGradThreads < nvec) p[c].load(row, (i + c * kGradThreads) * VW, 0.f);
  }
  __device__ void save(void* row, int i, int nvec) const {
#pragma unroll
    for (int c = 0; c < kParts; ++c)
      if (i + c * kGradThreads < nvec) p[c].save(static_cast<uint8_t*>(row), (i + c * kGradThreads) * VW);
  }
  __device__ void widen(float (&v)[kValues]) const {
#pragma unroll
    for (int c = 0; c < kParts; ++c) p[c].widen(reinterpret_cast<float(&)[VW]>(v[c * VW]));
  }
  __device__ void narrow(const float (&v)[kValues]) {
#pragma unroll
    for (int c = 0; c < kParts; ++c) p[c].narrow(reinterpret_cast<const float(&)[VW]>(v[c * VW]));
  }
};

// D zeros, 16 bytes at a time wherever the row begins, by a warp.
template <int kWbf16>
__device__ __forceinline__ void zero_row(uint8_t* row, int D) {
  constexpr int kElt = kWbf16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / kElt;
  const int whole = D > head ? (D - head) * kElt / 16 : 0;
  const int tail = head + whole * (16 / kElt);   // elements from here on, and before head, go alone
  auto one = [&](int i) {
    if (kWbf16) reinterpret_cast<uint16_t*>(row)[i] = 0;
    else reinterpret_cast<uint32_t*>(row)[i] = 0;
  };
  if (lane < head && lane < D) one(lane);
  if (tail + lane < D) one(tail + lane);
#pragma unroll 4
  for (int i = lane; i < whole; i += 32) reinterpret_cast<uint4*>(row + head * kElt)[i] = make_uint4(0, 0, 0, 0);
}

// CTAs [0, ranges * pieces): a range of the sorted order and a piece of the columns. The others (not
// accumulating): kZeroRows rows of dW each.
template <int kBf16, int kWbf16, int VW, int kAdd>
__global__ void __launch_bounds__(kGradThreads)
    embedding_grad_kernel(const void* dy, int64_t lddy, const uint32_t* ids, const uint32_t* perm, int N,
                          int V, int D, float scale, void* dW, int64_t ldw, float* part,
                          int ranges, int range, int pieces) {
  using In = RowPart<kBf16, VW>;
  using Out = RowPart<kWbf16, VW>;
  constexpr int kValues = In::kValues;
  __shared__ uint32_t s_id[kGradThreads], s_row[kGradThreads];
  __shared__ int s_absent[kZeroRows];
  start_next_launch();
  wait_for_launch_before();
  const int nvec = D / VW;
  if (static_cast<int>(blockIdx.x) >= ranges * pieces) {
    const int64_t row0 = (static_cast<int64_t>(blockIdx.x) - ranges * pieces) * kZeroRows;
    if (threadIdx.x < kZeroRows) {
      const int64_t v = row0 + threadIdx.x;
      int absent = 0;
      if (v < V) {
        const int at = lower_bound(ids, N, static_cast<uint32_t>(v));
        absent = at == N || ids[at] != static_cast<uint32_t>(v);
      }
      s_absent[threadIdx.x] = absent;
    }
    __syncthreads();
    for (int r = static_cast<int>(threadIdx.x >> 5); r < kZeroRows; r += kGradThreads / 32)
      if (s_absent[r]) zero_row<kWbf16>(static_cast<uint8_t*>(dW) + (row0 + r) * ldw * (kWbf16 ? 2 : 4), D);
    return;
  }
  const int r = static_cast<int>(blockIdx.x) / pieces;
  const int first = r * range;
  const int end = N - first < range ? N : first + range;
  const int i = static_cast<int>(blockIdx.x) % pieces * kGradThreads * In::kParts + static_cast<int>(threadIdx.x);
  // the ids on either side of the range (V: none)
  const uint32_t none = static_cast<uint32_t>(V);
  const uint32_t before = first > 0 ? ids[first - 1] : none;
  const uint32_t after = end < N ? ids[end] : none;
  float sum[kValues];
#pragma unroll
  for (int e = 0; e < kValues; ++e) sum[e] = 0.f;
  bool head = true;   // no id has ended yet in this range
  uint32_t id = none;
  auto row_of_id = [&](uint32_t row) { return static_cast<uint8_t*>(dW) + row * ldw * (kWbf16 ? 2 : 4); };
  auto end_of_id = [&](bool last, const Out& old) {
    if (id == none) return;
    if ((head && id == before) || (last && id == after)) {
      const int slot = head && id == before ? 0 : 1;
      RowPart<0, VW> out;
      out.narrow(sum);
      out.save(part + (static_cast<int64_t>(r) * 2 + slot) * D, i, nvec);
    } else {
      float v[kValues];
      if constexpr (kAdd) old.widen(v);
      finish_sum<kValues, kAdd>(sum, scale, v);
      Out out;
      out.narrow(sum);
      out.save(row_of_id(id), i, nvec);
    }
    head = false;
#pragma unroll
    for (int e = 0; e < kValues; ++e) sum[e] = 0.f;
  };
  // the old values of the rows that end: read with the rows of dy (adding)
  Out old[kAdd ? kAhead : 1], last_old;
  for (int at = first; at < end; at += kGradThreads) {
    const int n = end - at < kGradThreads ? end - at : kGradThreads;
    if (at > first) __syncthreads();
    if (static_cast<int>(threadIdx.x) < n) {
      s_id[threadIdx.x] = ids[at + threadIdx.x];
      s_row[threadIdx.x] = perm[at + threadIdx.x];
    }
    __syncthreads();
    for (int j = 0; j < n; j += kAhead) {
      In row[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (j + k < n && s_id[j + k] != none)
          row[k].load(static_cast<const uint8_t*>(dy) + s_row[j + k] * lddy * (kBf16 ? 2 : 4), i, nvec);
      if constexpr (kAdd) {
        uint32_t before_k = id;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (j + k >= n) break;
          const uint32_t here = s_id[j + k];
          if (here != before_k && here != none) old[k].load(row_of_id(here), i, nvec);
          before_k = here;
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (j + k >= n) break;
        const uint32_t here = s_id[j + k];
        if (here != id) {
          end_of_id(false, last_old);
          id = here;
          if constexpr (kAdd) last_old = old[k];
        }
        if (here != none) {
          float v[kValues];
          row[k].widen(v);
          add_n(sum, v);
        }
      }
    }
  }
  end_of_id(true, last_old);
}

// The ids that go on over the end of a range: the range in which one begins holds its first part in
// slot 1, the ranges after it the others in slot 0. CTA (range, piece of 128 vectors of columns, four a
// lane, so that few CTAs come for nothing), the parts dealt to its warps and added in a fixed order.
constexpr int kJoinWarps = 8;
constexpr int kJoinVectors = 4;

template <int kWbf16, int VW, int kAdd>
__global__ void __launch_bounds__(32 * kJoinWarps)
    embedding_join_kernel(const float* part, const uint32_t* ids, int N, int V, int D, float scale, void* dW,
                          int64_t ldw, int range, int pieces) {
  __shared__ __align__(16) float s_sum[kJoinWarps][32 * kJoinVectors * VW];
  __shared__ int s_last;
  wait_for_launch_before();
  const int r = static_cast<int>(blockIdx.x) / pieces;   // all ranges but the last
  const int first = r * range, end = first + range;
  const uint32_t id = ids[end - 1];
  if (id == static_cast<uint32_t>(V) || ids[end] != id) return;
  if (first > 0 && ids[first - 1] == id) return;   // it began in an earlier range
  if (threadIdx.x == 0) s_last = (lower_bound(ids, N, id + 1) - 1) / range;
  __syncthreads();
  const int last = s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int base = static_cast<int>(blockIdx.x) % pieces * 32 * kJoinVectors, nvec = D / VW;
  float sum[kJoinVectors][VW];
#pragma unroll
  for (int k = 0; k < kJoinVectors; ++k)
#pragma unroll
    for (int e = 0; e < VW; ++e) sum[k][e] = 0.f;
#pragma unroll 2
  for (int q = r + warp; q <= last; q += kJoinWarps) {
    const float* const from = part + (static_cast<int64_t>(q) * 2 + (q == r ? 1 : 0)) * D;
#pragma unroll
    for (int k = 0; k < kJoinVectors; ++k) {
      const int i = base + k * 32 + lane;
      if (i < nvec) {
        Param<0, VW> in;
        float v[VW];
        in.load(from, i * VW, 0.f);
        in.widen(v);
        add_n(sum[k], v);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kJoinVectors; ++k) {
    Param<0, VW> out;
    out.narrow(sum[k]);
    out.save(reinterpret_cast<uint8_t*>(s_sum[warp]), (k * 32 + lane) * VW);
  }
  __syncthreads();
  const int i = base + static_cast<int>(threadIdx.x);   // a vector a thread
  if (threadIdx.x >= 32 * kJoinVectors || i >= nvec) return;
  float total[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) total[e] = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    Param<0, VW> in;
    float v[VW];
    in.load(s_sum[w], static_cast<int>(threadIdx.x) * VW, 0.f);
    in.widen(v);
    add_n(total, v);
  }
  uint8_t* const row = static_cast<uint8_t*>(dW) + id * ldw * (kWbf16 ? 2 : 4);
  Param<kWbf16, VW> at;
  float old[VW];
  if constexpr (kAdd) {
    at.load(row, i * VW, 0.f);
    at.widen(old);
  }
  finish_sum<VW, kAdd>(total, scale, old);
  at.narrow(total);
  at.save(row, i * VW);
}

// f(VW) for the widest access: 8 elements, 4 or 1.
template <typename F>
cudaError_t with_width(int vw, F&& f) {
  if (vw >= 8) return f(std::integral_constant<int, 8>{});
  if (vw >= 4) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 1>{});
}

template <typename F>
cudaError_t with_types(int a, int b, F&& f) {
  using One = std::integral_constant<int, 1>;
  using Zero = std::integral_constant<int, 0>;
  if (a) return b ? f(One{}, One{}) : f(One{}, Zero{});
  return b ? f(Zero{}, One{}) : f(Zero{}, Zero{});
}

// Elements that both matrices allow at a time: rows of 16-byte accesses, or 8-byte ones (fp32's
// four at a time count as one of bf16's eight).
int common_width(int D, int bf16_a, int64_t lda, const void* a, int bf16_b, int64_t ldb, const void* b) {
  auto fits = [&](int v) {
    auto one = [&](int bf16, int64_t ld, const void* p) {
      const int elt = bf16 ? 2 : 4, bytes = v * elt < 16 ? v * elt : 16;
      return ld * elt % bytes == 0 && reinterpret_cast<uintptr_t>(p) % static_cast<unsigned>(bytes) == 0;
    };
    return D % v == 0 && one(bf16_a, lda, a) && one(bf16_b, ldb, b);
  };
  return fits(8) ? 8 : fits(4) ? 4 : 1;
}

}  // namespace

cudaError_t launch_embedding(const void* weight, int wbf16, int64_t ldw, const int32_t* tokens, int N,
                             int V, int D, float scale, int ignore_index, void* y, int bf16, int64_t ldy,
                             int32_t* status, cudaStream_t stream) {
  const int vw = common_width(D, wbf16, ldw, weight, bf16, ldy, y);
  return with_width(vw, [&](auto w) {
    constexpr int VW = w();
    const int nvec = D / VW;
    const int X = threads_of_row(N, nvec, lookup_vectors(VW), 8, kLookupThreads);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(N) * X + kLookupThreads - 1) / kLookupThreads),
                    static_cast<unsigned>((nvec + X * lookup_vectors(VW) - 1) / (X * lookup_vectors(VW))));
    return with_types(wbf16, bf16, [&](auto wb, auto b) {
      embedding_kernel<wb(), b(), VW><<<grid, kLookupThreads, 0, stream>>>(
          weight, ldw, tokens, N, V, nvec, scale, ignore_index, y, ldy, status, X);
      return cudaGetLastError();
    });
  });
}

cudaError_t launch_embedding_grad(const void* dy, int bf16, int64_t lddy, const uint32_t* ids,
                                  const uint32_t* perm, int N, int V, int D, float scale, void* dW, int wbf16,
                                  int64_t ldw, int accumulate, float* part, cudaStream_t stream) {
  const int range = embed_range(N), ranges = (N + range - 1) / range;
  const int vw = common_width(D, bf16, lddy, dy, wbf16, ldw, dW);
  const unsigned zeros = accumulate ? 0 : static_cast<unsigned>((static_cast<int64_t>(V) + kZeroRows - 1) / kZeroRows);
  return with_width(vw, [&](auto w) {
    constexpr int VW = w();
    const int nvec = D / VW;
    return with_types(bf16, wbf16, [&](auto b, auto wb) {
      auto go = [&](auto add) {
        const int piece = kGradThreads * row_parts(VW), pieces = (nvec + piece - 1) / piece;
        const unsigned grid = static_cast<unsigned>(ranges * pieces) + zeros;
        if (grid == 0) return cudaSuccess;
        const cudaError_t e =
            launch_after(embedding_grad_kernel<b(), wb(), VW, add()>, dim3(grid), dim3(kGradThreads), 0, stream, dy,
                         lddy, ids, perm, N, V, D, scale, dW, ldw, part, ranges, range, pieces);
        if (e != cudaSuccess || ranges <= 1) return e;
        const int columns = (nvec + 32 * kJoinVectors - 1) / (32 * kJoinVectors);
        return launch_after(embedding_join_kernel<wb(), VW, add()>,
                            dim3(static_cast<unsigned>((ranges - 1) * columns)), dim3(32 * kJoinWarps), 0, stream,
                            static_cast<const float*>(part), ids, N, V, D, scale, dW, ldw, range, columns);
      };
      return accumulate ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 0>{});
    });
  });
}

}  // namespace flce
