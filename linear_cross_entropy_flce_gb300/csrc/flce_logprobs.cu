// Log probabilities of given tokens over a logits matrix Z [N, V] (fp32 or bf16), with
// each row's entropy and most likely ids, and their gradient in the logits.
//
// Forward, two passes over each row: pass 1 takes the maximum, pass 2 sums 2^d and 2^d d
// against it (flce_rowstat.cuh) and collects the candidates of the ranking. Any element of
// the top k is at least as large as the k-th largest of 32 maxima over disjoint groups of
// threads, since those k groups hold k elements that large; pass 1 gives those maxima, so
// pass 2 only keeps the elements that reach that threshold, a few more than k on most
// logits. One warp sorts them. A row where too many reach it is ranked by k passes
// instead, each the largest key below the one before.
//
//   logprob_stream_kernel : rows of up to 832 KB. Persistent clusters of 1-8 CTAs, one row
//       at a time; each CTA's slice is copied into shared memory by the bulk-copy engine,
//       double-buffered, so both passes read shared memory and every logit leaves DRAM
//       once. Most of the CTA's warps do the passes; one sorts the candidates of the row
//       before, sends the CTA's part of it and starts the copies; one finds the ranking's
//       threshold while the sums are taken; one joins the parts of
//       the rows that are this CTA's (each row's meet in another CTA of the cluster), so
//       that none of it holds the passes up.
//       8192 x 128256 bf16 (2.1 GB, 309 us at the copy rate): 372 us (5.6 TB/s), with 5 alternatives
//       494, with 20 582; 4096 x 128256 fp32 293, 355, 381. Bound by the exponentials and maxima
//       beside the reads (two packed instructions for each pair of logits and pass), and with
//       alternatives by the second look at the threads whose maximum reaches the threshold.
//   logprob_warp_kernel : rows of up to 8 KB, one warp each: 16384 x 2000 bf16 16.7 us (3.9 TB/s).
//   logprob_rows_kernel : longer rows; one CTA each, read twice from global memory.
//
// Backward, elementwise: every entry of dZ from its logit and five numbers of its row. Bound by
// HBM: 8192 x 128256 bf16 590 us (7.1 TB/s), 4096 x 128256 fp32 590 us (7.1 TB/s).
//
// Rows may start at any element: the elements before the first 16-byte boundary and
// after the last one are read singly.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "flce_internal.h"
#include "ptx.cuh"
#include "flce_rowstat.cuh"
#include "flce_topk.cuh"

namespace flce {

namespace {

constexpr int kRowThreads = 512;
constexpr int kCandidates = 448;
constexpr int kMaxRowCluster = 8;

template <int kBf16>
struct Logit;

template <>
struct Logit<0> {
  static constexpr int E = 4, kBytes = 4;
  __device__ static float load1(const uint8_t* p) { return *reinterpret_cast<const float*>(p); }
  __device__ static void store1(uint8_t* p, float v) { *reinterpret_cast<float*>(p) = v; }
  __device__ static void widen(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  __device__ static uint4 narrow(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <>
struct Logit<1> {
  static constexpr int E = 8, kBytes = 2;
  __device__ static float load1(const uint8_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
  }
  __device__ static void store1(uint8_t* p, float v) {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(pack_bf16(v, 0.f) & 0xFFFFu);
  }
  __device__ static void widen(const uint4& w, float (&x)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(a[i] << 16);
      x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 narrow(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
  }
};

// Elements of a row before its first 16-byte boundary.
template <int kBf16>
__device__ __forceinline__ int row_head(const uint8_t* row, int V) {
  using L = Logit<kBf16>;
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / L::kBytes;
  const int head = mis ? L::E - mis : 0;
  return head < V ? head : V;
}

__device__ __forceinline__ void record_error(int32_t* status, int code) {
  if (status != nullptr) atomicCAS(reinterpret_cast<int*>(status), 0, code);
}

template <int kBf16, bool kTop>
__global__ void __launch_bounds__(kRowThreads)
    logprob_rows_kernel(const uint8_t* __restrict__ z, int64_t ld_bytes,
                        const int32_t* __restrict__ tokens, int N, int V, int ignore_index,
                        int top_k, float inv_t, float* __restrict__ logprob,
                        float* __restrict__ entropy, float* __restrict__ lse,
                        float* __restrict__ top_lp, int32_t* __restrict__ top_id,
                        int32_t* status) {
  using L = Logit<kBf16>;
  constexpr int E = L::E;
  constexpr int kWarps = kRowThreads / 32;
  __shared__ float s_group[32];       // maxima over groups of kRowThreads / 32 threads
  __shared__ float2 s_sum[kWarps];
  __shared__ uint64_t s_cand[kTop ? kCandidates : 1];
  __shared__ uint64_t s_best[kTop ? kWarps : 1];
  __shared__ uint64_t s_list[kTop ? kMaxTopK : 1];
  __shared__ int s_count;
  __shared__ float s_zt;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float c = kLog2e * inv_t;

  for (int row = blockIdx.x; row < N; row += gridDim.x) {
    if (tid == 0) s_count = 0;   // offers start after the next barrier
    const uint8_t* zr = z + static_cast<int64_t>(row) * ld_bytes;
    const int head = row_head<kBf16>(zr, V);
    const int nvec = (V - head) / E;
    const int tail = head + nvec * E;
    const uint4* vec = reinterpret_cast<const uint4*>(zr + static_cast<int64_t>(head) * L::kBytes);
    const int y = tokens != nullptr ? tokens[row] : ignore_index;
    const bool bad = y != ignore_index && (y < 0 || y >= V);
    const int yt = (y == ignore_index || bad) ? -1 : y;
    // this thread's edge element, if it has one: before the first or after the last vector
    const int n_edge = head + (V - tail);
    const int ie = tid < head ? tid : tail + tid - head;
    const float xe = tid < n_edge ? L::load1(zr + static_cast<int64_t>(ie) * L::kBytes) : -INFINITY;

    float m = xe;
#pragma unroll 4
    for (int v = tid; v < nvec; v += kRowThreads) {
      float x[E];
      L::widen(__ldg(vec + v), x);
#pragma unroll
      for (int e = 0; e < E; ++e) m = max_nan(m, x[e]);
    }
    {
      constexpr int kGroup = kRowThreads / 32;
      float g = m;
#pragma unroll
      for (int o = kGroup / 2; o > 0; o >>= 1) g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
      if (tid % kGroup == 0) s_group[tid / kGroup] = g;
    }
    __syncthreads();
    const float gm = s_group[lane];
    float M = gm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    float thr = INFINITY;
    if constexpr (kTop) {
      // the top_k-th largest of the 32 group maxima
      int rank = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float o = __shfl_sync(0xffffffffu, gm, j);
        rank += (o > gm || (o == gm && j < lane)) ? 1 : 0;
      }
      const unsigned at = __ballot_sync(0xffffffffu, rank == top_k - 1);
      thr = at ? __shfl_sync(0xffffffffu, gm, __ffs(at) - 1) : -INFINITY;
    }

    // pass 2
    float s = 0.f, t = 0.f;
    auto add = [&](float x) {
      const float d = row_exponent(x, M, c);
      const float e = exp2_approx(d);
      s += e;
      t = fmaf(e, d, t);
    };
    auto offer = [&](float x, int id) {
      if (x >= thr && x > -INFINITY) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kCandidates) s_cand[at] = rank_key(x, id);
      }
    };
    if (M > -INFINITY && M < INFINITY) {
      const bool mine = kTop && m >= thr;
#pragma unroll 2
      for (int v = tid; v < nvec; v += kRowThreads) {
        float x[E];
        L::widen(__ldg(vec + v), x);
        const int base = head + v * E;
        if (kTop && mine) {
#pragma unroll
          for (int e = 0; e < E; ++e) offer(x[e], base + e);
        }
        if (static_cast<unsigned>(yt - base) < static_cast<unsigned>(E)) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (base + e == yt) {
              s_zt = x[e];
              x[e] = -INFINITY;
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) add(x[e]);
      }
      if (tid < n_edge) {
        if (kTop) offer(xe, ie);
        if (ie == yt) s_zt = xe;
        else add(xe);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    if (lane == 0) s_sum[warp] = make_float2(s, t);
    __syncthreads();

    uint64_t list = 0;   // warp 0: the row's ranking, one key per lane
    if constexpr (kTop) {
      const int count = s_count;
      if (count <= kCandidates) {
        if (warp == 0) {
          for (int b = 0; b < count; b += 32) {
            uint64_t k = b + lane < count ? s_cand[b + lane] : 0;
            k = warp_sort_desc(k, lane);
            list = b == 0 ? k : warp_merge_desc(list, k, lane);
          }
        }
      } else {
        // too many reach the threshold: the largest key below the one before, k times
        uint64_t below = ~0ull;
        for (int i = 0; i < top_k; ++i) {
          uint64_t best = 0;
          auto look = [&](float x, int id) {
            if (x > -INFINITY) {
              const uint64_t k = rank_key(x, id);
              if (k < below && k > best) best = k;
            }
          };
          for (int v = tid; v < nvec; v += kRowThreads) {
            float x[E];
            L::widen(__ldg(vec + v), x);
#pragma unroll
            for (int e = 0; e < E; ++e) look(x[e], head + v * E + e);
          }
          if (tid < n_edge) look(xe, ie);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const uint64_t k = __shfl_xor_sync(0xffffffffu, best, o);
            best = k > best ? k : best;
          }
          if (lane == 0) s_best[warp] = best;
          __syncthreads();
          best = lane < kWarps ? s_best[lane] : 0;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const uint64_t k = __shfl_xor_sync(0xffffffffu, best, o);
            best = k > best ? k : best;
          }
          below = best;
          if (tid == 0) s_list[i] = best;
          __syncthreads();
          if (best == 0) {   // no id is left
            for (int j = i + 1 + tid; j < top_k; j += kRowThreads) s_list[j] = 0;
            __syncthreads();
            break;
          }
        }
        if (warp == 0) list = lane < top_k ? s_list[lane] : 0;
      }
    }
    if (warp == 0) {
      float2 p = lane < kWarps ? s_sum[lane] : make_float2(0.f, 0.f);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        p.x += __shfl_xor_sync(0xffffffffu, p.x, o);
        p.y += __shfl_xor_sync(0xffffffffu, p.y, o);
      }
      const RowOut r = row_finish(RowPart{M, p.x, p.y}, yt >= 0 ? s_zt : 0.f, yt >= 0, inv_t, c);
      if (lane == 0) {
        if (logprob != nullptr) logprob[row] = bad ? __uint_as_float(0x7FC00000u) : r.logprob;
        if (entropy != nullptr) entropy[row] = r.entropy;
        if (lse != nullptr) lse[row] = r.lse;
        if (bad) record_error(status, 8);
      }
      if constexpr (kTop) {
        if (lane < top_k) {
          const int64_t at = static_cast<int64_t>(row) * top_k + lane;
          const bool none = list == 0;
          top_id[at] = none ? -1 : key_id(list);
          top_lp[at] = r.lse != r.lse ? r.lse : none ? -INFINITY : id_logprob(r, key_value(list), inv_t);
        }
      }
    }
    __syncthreads();   // shared memory is reused by the next row
  }
}

// ---- rows through shared memory ----------------------------------------------------------

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void fadd2(float& d0, float& d1, float a0, float a1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}
// (d0, d1) = (a0, a1) * (b0, b1) + (c0, c1)
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b0, float b1,
                                      float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Running maximum over 16-byte vectors, bf16 two at a time.
template <int kBf16>
struct VecMax;
template <>
struct VecMax<1> {
  uint32_t a = 0xFF80FF80u, b = 0xFF80FF80u;   // -inf
  __device__ void take(const uint4& w) {
    a = max2_nan(a, max2_nan(w.x, w.y));
    b = max2_nan(b, max2_nan(w.z, w.w));
  }
  __device__ float value() const {
    const uint32_t m = max2_nan(a, b);
    return max_nan(lo_of(m), hi_of(m));
  }
};
template <>
struct VecMax<0> {
  float a = -INFINITY, b = -INFINITY;
  __device__ void take(const uint4& w) {
    a = max_nan(a, max_nan(__uint_as_float(w.x), __uint_as_float(w.y)));
    b = max_nan(b, max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  __device__ float value() const { return max_nan(a, b); }
};

// Maximum over the warp that keeps a NaN, in one instruction.
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// 32 values in descending order over the warp.
__device__ __forceinline__ float warp_sort_values(float v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
    const bool desc = (lane & size) == 0 || size == 32;
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, j);
      v = ((lane & j) == 0) == desc ? fmaxf(v, o) : fminf(v, o);
    }
  }
  return v;
}

// Whether a 16-byte vector has an element that reaches thr (a value of the row's type).
template <int kBf16>
struct Reaches;
template <>
struct Reaches<1> {
  uint32_t below;   // the bf16 value before thr, in both halves (-inf for -inf)
  __device__ explicit Reaches(float thr) {
    const uint32_t b = __float_as_uint(thr) >> 16;
    const uint32_t p = b == 0xFF80u ? b : (b & 0x7FFFu) == 0 ? 0x8001u : (b & 0x8000u) ? b + 1 : b - 1;
    below = p | (p << 16);
  }
  __device__ bool operator()(const uint4& w) const {
    return max2_nan(max2_nan(max2_nan(w.x, w.y), max2_nan(w.z, w.w)), below) != below;
  }
};
template <>
struct Reaches<0> {
  float thr;
  __device__ explicit Reaches(float t) : thr(t) {}
  __device__ bool operator()(const uint4& w) const {
    const float m = fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                          fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    return m >= thr && m > -INFINITY;
  }
};

// Sums 2^d and 2^d d over 16-byte vectors of a row with maximum M.
template <int kBf16>
struct RowSums {
  float M, c, ref, lo;
  uint32_t lo2;
  bool clamp;   // element by element, without a reference or a floor
  float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
  // Smaller logits (and -inf) are raised to a floor: far enough below M that their 2^d is 0,
  // near enough that d is finite. In bf16 rows of logits of 1e4 or more rounding may leave
  // no such value: those clamp the exponents.
  // reach: 200 / c
  __device__ RowSums(float m, float cc, float reach) : M(m), c(cc), ref(row_ref(m, cc)) {
    const float below = m - reach;
    asm("cvt.rz.bf16x2.f32 %0, %1, %1;" : "=r"(lo2) : "f"(below));
    lo = kBf16 ? lo_of(lo2) : below;
    clamp = !has_ref(m, cc) || !(fmaf(lo, cc, -ref) < -150.f);
  }
  __device__ void add(uint4 w) {
    constexpr int E = Logit<kBf16>::E;
    float x[E];
    if (!clamp) {
      if constexpr (kBf16) {
        w.x = max2_nan(w.x, lo2);
        w.y = max2_nan(w.y, lo2);
        w.z = max2_nan(w.z, lo2);
        w.w = max2_nan(w.w, lo2);
      }
      Logit<kBf16>::widen(w, x);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        if constexpr (!kBf16) {
          x[e] = fmaxf(x[e], lo);
          x[e + 1] = fmaxf(x[e + 1], lo);
        }
        ffma2(x[e], x[e + 1], x[e], x[e + 1], c, c, -ref, -ref);
      }
    } else {
      Logit<kBf16>::widen(w, x);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = row_exponent(x[e], M, c);
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float e0 = exp2_approx(x[e]), e1 = exp2_approx(x[e + 1]);
      fadd2(s0, s1, e0, e1);
      ffma2(t0, t1, e0, e1, x[e], x[e + 1], t0, t1);
    }
  }
  __device__ void add_one(float z) {
    const float d = row_exponent(z, M, c), e = exp2_approx(d);
    s0 += e;
    t0 = fmaf(e, d, t0);
  }
};

// Element e of a 16-byte vector.
template <int kBf16>
__device__ __forceinline__ float element_of(const uint4& w, int e) {
  const int i = kBf16 ? e >> 1 : e;
  const uint32_t a = i & 1 ? w.y : w.x, b = i & 1 ? w.w : w.z;
  const uint32_t v = i & 2 ? b : a;
  return kBf16 ? (e & 1 ? hi_of(v) : lo_of(v)) : __uint_as_float(v);
}

template <int kBf16>
__device__ __forceinline__ uint4 no_logits() {
  const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;   // -inf
  return make_uint4(none, none, none, none);
}

// ---- short rows: one warp each -----------------------------------------------------------
//
// The row stays in the warp's registers for both passes: no barriers, and the lanes' maxima
// are the 32 groups of the ranking's threshold.
constexpr int kWarpRowWarps = 4;
constexpr int kWarpCandidates = 96;

template <int kBf16, bool kTop, int kNv>
__global__ void __launch_bounds__(kWarpRowWarps * 32)
    logprob_warp_kernel(const uint8_t* __restrict__ z, int64_t ld_bytes,
                        const int32_t* __restrict__ tokens, int N, int V, int ignore_index,
                        int top_k, float inv_t, float* __restrict__ logprob,
                        float* __restrict__ entropy, float* __restrict__ lse,
                        float* __restrict__ top_lp, int32_t* __restrict__ top_id,
                        int32_t* status) {
  using L = Logit<kBf16>;
  constexpr int E = L::E;
  __shared__ uint64_t s_cand[kTop ? kWarpRowWarps : 1][kTop ? kWarpCandidates : 1];
  __shared__ int s_count[kWarpRowWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kWarpRowWarps + warp;
  if (row >= N) return;
  const float c = kLog2e * inv_t;
  const uint8_t* zr = z + static_cast<int64_t>(row) * ld_bytes;
  const int head = row_head<kBf16>(zr, V);
  const int nvec = (V - head) / E;
  const int tail = head + nvec * E;
  const uint4* vec = reinterpret_cast<const uint4*>(zr + static_cast<int64_t>(head) * L::kBytes);
  uint4 w[kNv];
#pragma unroll
  for (int j = 0; j < kNv; ++j) w[j] = lane + 32 * j < nvec ? __ldg(vec + lane + 32 * j) : no_logits<kBf16>();
  const int ie = lane < head ? lane : lane < head + V - tail ? tail + lane - head : -1;
  const float xe = ie >= 0 ? L::load1(zr + static_cast<int64_t>(ie) * L::kBytes) : -INFINITY;
  const int y = tokens != nullptr ? tokens[row] : ignore_index;
  const bool bad = y != ignore_index && (y < 0 || y >= V);
  const int yt = (y == ignore_index || bad) ? -1 : y;
  VecMax<kBf16> vm;
#pragma unroll
  for (int j = 0; j < kNv; ++j) vm.take(w[j]);
  const float mine = max_nan(vm.value(), xe);
  const float M = warp_max_nan(mine);
  RowPart part{M, 0.f, 0.f};
  float zt = 0.f;
  uint64_t list = 0;
  if (M > -INFINITY && M < INFINITY) {
    if constexpr (kTop) {
      const float thr = __shfl_sync(0xffffffffu, warp_sort_values(mine, lane), top_k - 1);
      const Reaches<kBf16> reaches(thr);
      uint32_t hit = 0;   // this lane's vectors that reach the threshold: a few in the warp
#pragma unroll
      for (int j = 0; j < kNv; ++j) hit |= (reaches(w[j]) ? 1u : 0u) << j;
      if (lane == 0) s_count[warp] = 0;
      __syncwarp();
      auto offer = [&](float x, int id) {
        if (x >= thr && x > -INFINITY) {
          const int at = atomicAdd(&s_count[warp], 1);
          if (at < kWarpCandidates) s_cand[warp][at] = rank_key(x, id);
        }
      };
      for (; hit != 0; hit &= hit - 1) {
        const int v = lane + 32 * (__ffs(hit) - 1);
        const uint4 again = __ldg(vec + v);   // (indexing the registers would move them to memory)
        float x[E];
        L::widen(again, x);
        uint32_t in = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) in |= (x[e] >= thr && x[e] > -INFINITY ? 1u : 0u) << e;
        int at = atomicAdd(&s_count[warp], __popc(in));
        for (; in != 0; in &= in - 1, ++at) {
          const int e = __ffs(in) - 1;
          if (at < kWarpCandidates) s_cand[warp][at] = rank_key(element_of<kBf16>(again, e), head + v * E + e);
        }
      }
      if (ie >= 0) offer(xe, ie);
      __syncwarp();
      const int count = s_count[warp];
      if (count <= kWarpCandidates) {
        for (int b = 0; b < count; b += 32) {
          const uint64_t key = warp_sort_desc(b + lane < count ? s_cand[warp][b + lane] : 0, lane);
          list = b == 0 ? key : warp_merge_desc(list, key, lane);
        }
      } else {
        // too many equal ones: the largest key below the one before, top_k times
        uint64_t below = ~0ull;
        for (int i = 0; i < top_k && below != 0; ++i) {
          uint64_t best = 0;
          auto look = [&](float x, int id) {
            const uint64_t key = x > -INFINITY ? rank_key(x, id) : 0;
            if (key < below && key > best) best = key;
          };
          for (int v = lane; v < nvec; v += 32) {
            const uint4 again = __ldg(vec + v);
            for (int e = 0; e < E; ++e) look(element_of<kBf16>(again, e), head + v * E + e);
          }
          if (ie >= 0) look(xe, ie);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const uint64_t key = __shfl_xor_sync(0xffffffffu, best, o);
            best = key > best ? key : best;
          }
          below = best;
          if (lane == i) list = best;
        }
      }
    }
    // the token's element leaves the sums
    bool own = ie >= 0 && ie == yt;
    if (own) zt = xe;
    RowSums<kBf16> sums(M, c, 200.f / c);
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
      const int base = head + (lane + 32 * j) * E;
      if (yt >= 0 && static_cast<unsigned>(yt - base) < static_cast<unsigned>(E) && yt < tail) {
        float x[E];
        L::widen(w[j], x);
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (base + e == yt) {
            zt = x[e];
            x[e] = -INFINITY;
          }
        w[j] = L::narrow(x);
        own = true;
      }
      sums.add(w[j]);
    }
    if (ie >= 0 && ie != yt) sums.add_one(xe);
    const unsigned who = __ballot_sync(0xffffffffu, own);
    zt = who ? __shfl_sync(0xffffffffu, zt, __ffs(who) - 1) : 0.f;
    part.s = sums.s0 + sums.s1;
    part.t = sums.t0 + sums.t1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      part.s += __shfl_xor_sync(0xffffffffu, part.s, o);
      part.t += __shfl_xor_sync(0xffffffffu, part.t, o);
    }
  }
  const RowOut r = row_finish(part, zt, yt >= 0, inv_t, c);
  if (lane == 0) {
    if (logprob != nullptr) logprob[row] = bad ? __uint_as_float(0x7FC00000u) : r.logprob;
    if (entropy != nullptr) entropy[row] = r.entropy;
    if (lse != nullptr) lse[row] = r.lse;
    if (bad) record_error(status, 8);
  }
  if (kTop && lane < top_k) {
    const int64_t at = static_cast<int64_t>(row) * top_k + lane;
    const bool none = list == 0;
    top_id[at] = none ? -1 : key_id(list);
    top_lp[at] = r.lse != r.lse ? r.lse : none ? -INFINITY : id_logprob(r, key_value(list), inv_t);
  }
}

// ---- longer rows: clusters, through shared memory -------------------------------------------

// In place of a row's maximum: a CTA's wait ran out of time. (Maxima have no such NaN.)
constexpr uint32_t kLateMark = 0x7FC0A7E5u;

// What a CTA knows of a row: maximum, sums, the token's logit if it is in its slice (0
// otherwise), and its ranking.
struct __align__(16) RowMsg {
  float4 part;   // m, s, t, zt
  uint64_t list[kMaxTopK];
};

template <int kBf16, bool kTop, int kWarps, int kSlice, int kMinBlocks>
__global__ void __launch_bounds__((kWarps + 3) * 32, kMinBlocks)
    logprob_stream_kernel(const uint8_t* __restrict__ z, int64_t ld_bytes,
                          const int32_t* __restrict__ tokens, int N, int V, int ignore_index,
                          int top_k, float inv_t, float* __restrict__ logprob,
                          float* __restrict__ entropy, float* __restrict__ lse,
                          float* __restrict__ top_lp, int32_t* __restrict__ top_id,
                          int32_t* status, uint64_t timeout_ns) {
  using L = Logit<kBf16>;
  constexpr int E = L::E;
  constexpr int kData = kWarps * 32;          // threads that do the passes
  constexpr int kAll = kData + 32;            // and the warp that ranks
  constexpr int kBarMax = 1;   // named barriers; the others in pairs
  constexpr int kBarDone = 2, kBarFree = 4, kBarLanes = 6, kBarThr = 8;
  extern __shared__ __align__(128) uint8_t s_rows[];       // two slices
  __shared__ __align__(8) uint64_t s_full[2];   // a slice's copy has landed
  // A row's parts meet in one CTA, each in turn (row it of the cluster in CTA it % csize, its
  // turn u = it / csize): messages and their barriers alternate between turns.
  __shared__ __align__(8) uint64_t s_got[2];                    // every CTA's message is here
  __shared__ __align__(8) uint64_t s_used[kMaxRowCluster][2];   // CTA r has read this one's message
  __shared__ RowMsg s_msg[2][kMaxRowCluster];
  __shared__ float s_max[2][kWarps];            // each warp's maximum
  __shared__ float s_lanes[kTop ? 2 : 1][kWarps][kTop ? 32 : 1];   // each thread's
  __shared__ float s_thr[2];                    // the ranking's threshold
  __shared__ uint16_t s_hot[kTop ? 2 : 1][kTop ? kData : 1];   // the threads whose maximum reaches it
  __shared__ int s_nhot[2];
  __shared__ int s_ties[2];                     // whether many elements may be equal to it
  __shared__ float2 s_sum[2][kWarps];
  __shared__ float s_m[2], s_zt[2];
  __shared__ int s_count[2];
  __shared__ uint64_t s_cand[kTop ? 2 : 1][kTop ? kCandidates : 1];
  // A wait ran out of time. From then on the CTA starts no copy (the slot's last one may still
  // be on its way), its rows are NaN, and a warp that waited for a peer in vain touches no
  // barrier of the exchange again: a phase that has not ended takes no second arrival.
  __shared__ volatile int s_late;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int crank = static_cast<int>(cluster_ctarank()), csize = static_cast<int>(cluster_size());
  const int first = static_cast<int>(blockIdx.x) / csize, step = static_cast<int>(gridDim.x) / csize;
  const float c = kLog2e * inv_t;
  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&s_full[k]), 1);
      mbar_init(smem_u32(&s_got[k]), 1);
      for (int r = 0; r < kMaxRowCluster; ++r) mbar_init(smem_u32(&s_used[r][k]), 1);
      s_count[k] = 0;
      s_zt[k] = 0.f;
    }
    s_late = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (csize > 1) cluster_sync();   // the barriers exist before a peer arrives on them

  const volatile int never = 0;
  int begun[2] = {0, 0};   // lane 0 of the last warp: turns of s_full begun

  // This CTA's slice of a row: vectors [v0, v0 + nv) of those between the row's first and
  // last 16-byte boundary; the first CTA has the elements before them, the last those after.
  struct Slice {
    const uint8_t* row;
    int head, tail, v0, nv;
  };
  auto slice_at = [&](const uint8_t* at) {
    Slice q;
    q.row = at;
    q.head = row_head<kBf16>(at, V);
    const int nvec = (V - q.head) / E;
    q.tail = q.head + nvec * E;
    const int per = (nvec + csize - 1) / csize;
    q.v0 = min(nvec, crank * per);
    q.nv = min(nvec, q.v0 + per) - q.v0;
    return q;
  };
  const Slice q_first = slice_at(z);
  const bool alike = ld_bytes % 16 == 0;   // every row starts as the first does
  auto slice_of = [&](int row) {
    const uint8_t* at = z + static_cast<int64_t>(row) * ld_bytes;
    if (!alike) return slice_at(at);
    Slice q = q_first;
    q.row = at;
    return q;
  };
  // single element number i of this CTA (a few at most): its id, or -1
  auto single_of = [&](const Slice& q, int i) {
    const int n_head = crank == 0 ? q.head : 0, n_tail = crank == csize - 1 ? V - q.tail : 0;
    return i < n_head ? i : i < n_head + n_tail ? q.tail + i - n_head : -1;
  };

  // Writes a row's outputs from its joined part; the whole warp calls.
  auto finish = [&](int row, int y, const RowPart& part, float zt, uint64_t list, bool late) {
    const bool bad = y != ignore_index && (y < 0 || y >= V);
    RowOut r = row_finish(part, zt, y != ignore_index && !bad, inv_t, c);
    const float nan = __uint_as_float(0x7FC00000u);
    if (late) r.logprob = r.entropy = r.lse = nan;
    if (lane == 0) {
      if (logprob != nullptr) logprob[row] = bad ? nan : r.logprob;
      if (entropy != nullptr) entropy[row] = r.entropy;
      if (lse != nullptr) lse[row] = r.lse;
      if (bad) record_error(status, 8);
      if (late) record_error(status, kStatusTimeout);
    }
    if (kTop && lane < top_k) {
      const int64_t at = static_cast<int64_t>(row) * top_k + lane;
      const bool none = list == 0;
      top_id[at] = none || late ? -1 : key_id(list);
      top_lp[at] = r.lse != r.lse ? r.lse : none ? -INFINITY : id_logprob(r, key_value(list), inv_t);
    }
  };

  if (warp < kWarps) {
    const float reach = 200.f / c;
    auto token_of = [&](int64_t row) {
      return tokens != nullptr && row < N ? tokens[row] : ignore_index;
    };
    int y_next = token_of(first);   // read a row ahead
    int it = 0;
    for (int row = first; row < N; row += step, ++it) {
      const int k = it & 1;
      const Slice q = slice_of(row);
      const int y = y_next;
      y_next = token_of(static_cast<int64_t>(row) + step);
      const int yt = (y == ignore_index || y < 0 || y >= V) ? -1 : y;
      const int ie = tid < 16 ? single_of(q, tid) : -1;
      const float xe = ie >= 0 ? L::load1(q.row + static_cast<int64_t>(ie) * L::kBytes) : -INFINITY;
      uint8_t* const buf = s_rows + k * kSlice;
      const uint4* const vec = reinterpret_cast<const uint4*>(buf);
      if (!mbar_wait_bounded(smem_u32(&s_full[k]), static_cast<uint32_t>((it >> 1) & 1), timeout_ns,
                             &s_late))
        s_late = 1;
      // pass 1
      VecMax<kBf16> vm;
#pragma unroll 4
      for (int v = tid; v < q.nv; v += kData) vm.take(vec[v]);
      const float mine = max_nan(vm.value(), xe);
      if constexpr (kTop) {
        s_lanes[k][warp][lane] = mine;
        __syncwarp();
        bar_arrive(kBarLanes + k, kAll);
      }
      const float wm = warp_max_nan(mine);
      if (lane == 0) s_max[k][warp] = wm;
      // the token's element: its thread keeps the value and takes it out of the sums
      const int id0 = q.head + q.v0 * E;   // id of the slice's first vector element
      float zt = 0.f;
      const bool taken = yt >= id0 && yt < id0 + q.nv * E && (yt - id0) / E % kData == tid;
      const bool own = taken || (ie >= 0 && ie == yt);
      if (own) zt = xe;
      if (taken) {
        uint8_t* at = buf + static_cast<int64_t>(yt - id0) * L::kBytes;
        zt = L::load1(at);
        if (kBf16) *reinterpret_cast<uint16_t*>(at) = 0xFF80u;   // -inf
        else *reinterpret_cast<float*>(at) = -INFINITY;
      }
      bar_sync(kBarMax, kData);
      const float M = warp_max_nan(s_max[k][lane % kWarps]);
      // the last warp has taken what this slot held
      if (it >= 2) bar_sync(kBarFree + k, kAll);
      if (own) s_zt[k] = zt;
      float s = 0.f, t = 0.f;
      if (M > -INFINITY && M < INFINITY) {
        RowSums<kBf16> sums(M, c, reach);
#pragma unroll 2
        for (int v = tid; v < q.nv; v += kData) sums.add(vec[v]);
        if (ie >= 0 && ie != yt) sums.add_one(xe);
        s = sums.s0 + sums.s1;
        t = sums.t0 + sums.t1;
      }
      if constexpr (kTop) {
        // the candidates: from the threads whose maximum reaches the threshold
        bar_sync(kBarThr + k, kAll);
        const float thr = s_thr[k];
        const bool live = M > -INFINITY && M < INFINITY;
        auto offer_one = [&](float x, int id) {
          if (x >= thr && x > -INFINITY) {
            const int at = atomicAdd(&s_count[k], 1);
            if (at < kCandidates) s_cand[k][at] = rank_key(x, id);
          }
        };
        int equal = 0;   // of this warp: elements equal to the threshold so far
        // Many equal ones: only the first top_k of them count, of this warp too, so that the
        // list holds what eight warps offer. The whole warp calls.
        auto offer_first = [&](const uint4& w, int id) {
          float x[E];
          L::widen(w, x);
          uint32_t gt = 0, eq = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            gt |= (x[e] > thr ? 1u : 0u) << e;
            eq |= (x[e] == thr && x[e] > -INFINITY ? 1u : 0u) << e;
          }
          int before = __popc(eq);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int p = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += p;
          }
          const int room = max(top_k - equal - (before - __popc(eq)), 0);   // of this lane's
          equal += __shfl_sync(0xffffffffu, before, 31);
          while (__popc(eq) > room) eq &= ~(0x80000000u >> __clz(eq));
          for (uint32_t in = gt | eq; in != 0; in &= in - 1) {
            const int e = __ffs(in) - 1;
            offer_one(element_of<kBf16>(w, e), id + e);
          }
        };
        if (live) {
          const Reaches<kBf16> reaches(thr);
          if (s_ties[k]) {
            for (int vw = warp * 32; vw < q.nv; vw += kData) {
              const uint4 w = vw + lane < q.nv ? vec[vw + lane] : no_logits<kBf16>();
              if (__any_sync(0xffffffffu, reaches(w))) offer_first(w, id0 + (vw + lane) * E);
            }
          } else {
            // the vectors of the threads whose maximum reaches it, dealt to the whole CTA: left
            // to those threads (or their warps) their chain of loads holds up the others
            const int hot = s_nhot[k];
            const int shift = hot > 1 ? 32 - __clz(hot - 1) : 0;
            const int rounds = (q.nv + kData - 1) / kData;
            for (int i = tid; i < rounds << shift; i += kData) {
              const int h = i & ((1 << shift) - 1);
              const int v = h < hot ? s_hot[k][h] + (i >> shift) * kData : q.nv;
              if (v < q.nv) {
                const uint4 w = vec[v];
                if (reaches(w)) {   // one reservation for all of the vector's
                  float x[E];
                  L::widen(w, x);
                  uint32_t in = 0;
#pragma unroll
                  for (int e = 0; e < E; ++e) in |= (x[e] >= thr && x[e] > -INFINITY ? 1u : 0u) << e;
                  int at = atomicAdd(&s_count[k], __popc(in));
                  for (; in != 0; in &= in - 1, ++at) {
                    const int e = __ffs(in) - 1;
                    if (at < kCandidates) s_cand[k][at] = rank_key(element_of<kBf16>(w, e), id0 + v * E + e);
                  }
                }
              }
            }
          }
          // the single elements, and the token's that the slice no longer holds
          if (ie >= 0) offer_one(xe, ie);
          if (taken) offer_one(zt, yt);
        }
        __syncwarp();
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
      }
      if (lane == 0) s_sum[k][warp] = make_float2(s, t);
      if (tid == 0) s_m[k] = M;
      bar_arrive(kBarDone + k, kAll);
    }
  } else if (warp == kWarps) {
    auto copy = [&](int row, int k) {
      const Slice q = slice_of(row);
      const uint32_t bytes = static_cast<uint32_t>(q.nv) * 16u, bar = smem_u32(&s_full[k]);
      ++begun[k];
      if (bytes == 0) {   // the row has no vector here: its turn of the barrier passes all the same
        mbar_arrive(bar);
        return;
      }
      const uint8_t* src = q.row + static_cast<int64_t>(q.head) * L::kBytes + static_cast<int64_t>(q.v0) * 16;
      const uint32_t dst = smem_u32(s_rows + k * kSlice);
      // the passes' reads and writes of the buffer come before the copy's
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive_expect_tx(bar, bytes);
      for (uint32_t off = 0; off < bytes; off += 16384u) {
        const uint32_t n = min(16384u, bytes - off);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                dst + off),
            "l"(src + off), "r"(n), "r"(bar)
            : "memory");
      }
    };
    if (lane == 0) {
      if (first < N) copy(first, 0);
      if (first + step < N) copy(first + step, 1);
    }
    bool sending = true;   // of this lane
    int it = 0;
    for (int row = first; row < N; row += step, ++it) {
      const int k = it & 1;
      const bool more = row + 2 * static_cast<int64_t>(step) < N;
      const int y = tokens != nullptr ? tokens[row] : ignore_index;
      bar_sync(kBarDone + k, kAll);
      // take what the slot holds, start the copy into it and give it back, then sort
      const int count = kTop ? s_count[k] : 0;
      const bool copying = more && !s_late;
      float2 sums = lane < kWarps ? s_sum[k][lane] : make_float2(0.f, 0.f);
      RowPart part{s_m[k], 0.f, 0.f};
      float zt = s_zt[k];
      uint64_t list = 0;
      auto give_back = [&]() {
        __syncwarp();
        if (lane == 0) {
          s_count[k] = 0;
          s_zt[k] = 0.f;
          if (copying) copy(row + 2 * step, k);
        }
        __syncwarp();
        if (more) bar_arrive(kBarFree + k, kAll);
      };
      if (count <= 64) {
        uint64_t a = 0, b = 0;
        if constexpr (kTop) {
          if (lane < count) a = s_cand[k][lane];
          if (lane + 32 < count) b = s_cand[k][lane + 32];
        }
        give_back();
        if constexpr (kTop) {
          list = warp_sort_desc(a, lane);
          if (count > 32) list = warp_merge_desc(list, warp_sort_desc(b, lane), lane);
        }
      } else if (count <= kCandidates) {
        if constexpr (kTop) {
          for (int b = 0; b < count; b += 32) {
            const uint64_t key = warp_sort_desc(b + lane < count ? s_cand[k][b + lane] : 0, lane);
            list = b == 0 ? key : warp_merge_desc(list, key, lane);
          }
        }
        give_back();
      } else {
        // too many reach the threshold: the largest key below the one before, top_k times.
        // The token's element was taken out of the slice: it joins from its value.
        const Slice q = slice_of(row);
        const uint4* vec = reinterpret_cast<const uint4*>(s_rows + k * kSlice);
        const int id0 = q.head + q.v0 * E;
        const int ie = lane < 16 ? single_of(q, lane) : -1;
        const float xe = ie >= 0 ? L::load1(q.row + static_cast<int64_t>(ie) * L::kBytes) : -INFINITY;
        const bool mine = y != ignore_index && y >= id0 && y < id0 + q.nv * E;
        uint64_t below = ~0ull;
        for (int i = 0; i < top_k && below != 0; ++i) {
          uint64_t best = 0;
          auto look = [&](float x, int id) {
            if (x > -INFINITY) {
              const uint64_t key = rank_key(x, id);
              if (key < below && key > best) best = key;
            }
          };
          for (int v = lane; v < q.nv; v += 32) {
            float x[E];
            L::widen(vec[v], x);
#pragma unroll
            for (int e = 0; e < E; ++e) look(x[e], id0 + v * E + e);
          }
          if (ie >= 0) look(xe, ie);
          if (mine && lane == 31) look(zt, y);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const uint64_t key = __shfl_xor_sync(0xffffffffu, best, o);
            best = key > best ? key : best;
          }
          below = best;
          if (lane == i) list = best;
        }
        give_back();
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sums.x += __shfl_xor_sync(0xffffffffu, sums.x, o);
        sums.y += __shfl_xor_sync(0xffffffffu, sums.y, o);
      }
      part.s = sums.x;
      part.t = sums.y;

      if (csize == 1) {
        finish(row, y, part, zt, list, s_late != 0);
      } else {
        // to this row's CTA, once it has read the message of two turns before
        const int leader = it % csize, u = it / csize, slot = u & 1;
        if (u >= 2 && !mbar_wait_bounded<true>(smem_u32(&s_used[leader][slot]),
                                               static_cast<uint32_t>(((u >> 1) - 1) & 1),
                                               sending ? timeout_ns : 0, &never)) {
          sending = false;
          s_late = 1;
        }
        // asynchronous stores, counted in bytes on the receiver's barrier: no fence
        const uint32_t msg = mapa_shared(smem_u32(&s_msg[slot][crank]), static_cast<uint32_t>(leader));
        const uint32_t bar = mapa_shared(smem_u32(&s_got[slot]), static_cast<uint32_t>(leader));
        if (s_late) part.m = __uint_as_float(kLateMark);   // a row that came to nothing
        if (sending && lane == 0)
          asm volatile(
              "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(msg),
              "f"(part.m), "f"(part.s), "f"(part.t), "f"(zt), "r"(bar)
              : "memory");
        if (kTop && sending && lane < top_k)
          asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                           msg + 16u + 8u * lane),
                       "l"(list), "r"(bar)
                       : "memory");
      }
    }
  } else if (kTop && warp == kWarps + 1) {
    // the top_k-th largest of the maxima over the threads of equal lane
    int it = 0;
    for (int64_t row = first; row < N; row += step, ++it) {
      const int k = it & 1;
      bar_sync(kBarLanes + k, kAll);
      float each[kWarps], m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        each[w] = s_lanes[k][w][lane];
        m = fmaxf(m, each[w]);
      }
      const float thr = __shfl_sync(0xffffffffu, warp_sort_values(m, lane), top_k - 1);
      const int same = __popc(__ballot_sync(0xffffffffu, m == thr && thr > -INFINITY));
      int hot = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const unsigned in = __ballot_sync(0xffffffffu, each[w] >= thr && each[w] > -INFINITY);
        if (in >> lane & 1u)
          s_hot[k][hot + __popc(in & ((1u << lane) - 1u))] = static_cast<uint16_t>(w * 32 + lane);
        hot += __popc(in);
      }
      if (lane == 0) {
        s_thr[k] = thr;
        s_ties[k] = same > 4;
        s_nhot[k] = hot;
      }
      __syncwarp();
      bar_arrive(kBarThr + k, kAll);
    }
  } else if (csize > 1) {
    // joins the rows whose turn this CTA is
    bool waiting = true;
    int u = 0;
    for (int64_t row = first + static_cast<int64_t>(crank) * step; row < N;
         row += static_cast<int64_t>(csize) * step, ++u) {
      const int slot = u & 1;
      const int y = tokens != nullptr ? tokens[row] : ignore_index;
      RowPart part{-INFINITY, 0.f, 0.f};
      float zt = 0.f;
      uint64_t list = 0;
      if (waiting) {
        if (lane == 0)
          mbar_arrive_expect_tx(smem_u32(&s_got[slot]),
                                static_cast<uint32_t>(csize) * (16u + (kTop ? 8u * top_k : 0u)));
        __syncwarp();
        waiting = mbar_wait_bounded<true>(smem_u32(&s_got[slot]), static_cast<uint32_t>((u >> 1) & 1),
                                          timeout_ns, &never);
        waiting = __all_sync(0xffffffffu, waiting);
        if (!waiting) {
          // No CTA sends more than two messages that are not read: those land before the memory
          // is given back.
          s_late = 1;
          if (lane == 0) {
            const int64_t next = row + static_cast<int64_t>(csize) * step;
            if (next < N)
              mbar_arrive_expect_tx(smem_u32(&s_got[slot ^ 1]),
                                    static_cast<uint32_t>(csize) * (16u + (kTop ? 8u * top_k : 0u)));
            for (int d = 0; d < (next < N ? 2 : 1); ++d)
              mbar_wait_bounded<true>(smem_u32(&s_got[(u + d) & 1]), static_cast<uint32_t>(((u + d) >> 1) & 1),
                                      1000000000ull, &never);
          }
          __syncwarp();
        }
      }
      bool late = !waiting;
      if (waiting) {
        // lane r joins CTA r's sums; the rankings one after the other
        if (lane < csize) {
          const float4 p = s_msg[slot][lane].part;
          part = RowPart{p.x, p.y, p.z};
          zt = p.w;
          late = __float_as_uint(p.x) == kLateMark;
        }
#pragma unroll
        for (int o = kMaxRowCluster / 2; o > 0; o >>= 1) {
          const RowPart q{__shfl_xor_sync(0xffffffffu, part.m, o), __shfl_xor_sync(0xffffffffu, part.s, o),
                          __shfl_xor_sync(0xffffffffu, part.t, o)};
          row_join(part, q, c);
          zt += __shfl_xor_sync(0xffffffffu, zt, o);
        }
        part = RowPart{__shfl_sync(0xffffffffu, part.m, 0), __shfl_sync(0xffffffffu, part.s, 0),
                       __shfl_sync(0xffffffffu, part.t, 0)};
        zt = __shfl_sync(0xffffffffu, zt, 0);
        if constexpr (kTop) {
          for (int r = 0; r < csize; ++r) {
            const uint64_t key = lane < top_k ? s_msg[slot][r].list[lane] : 0;
            list = r == 0 ? key : warp_merge_desc(list, key, lane);
          }
        }
        __syncwarp();
        if (lane < csize)
          mbar_arrive_cluster(mapa_shared(smem_u32(&s_used[crank][slot]), static_cast<uint32_t>(lane)));
      }
      finish(static_cast<int>(row), y, part, zt, list, __any_sync(0xffffffffu, late || s_late != 0));
    }
  }
  // copies that nobody waited for land before the memory is given back (only after a timeout)
  if (warp == kWarps && lane == 0 && s_late) {
    for (int k = 0; k < 2; ++k)
      if (begun[k] > 0)
        mbar_wait_bounded(smem_u32(&s_full[k]), static_cast<uint32_t>((begun[k] - 1) & 1), 1000000000ull, &never);
  }
  __syncwarp();
  // no CTA leaves while a peer may still write to it or arrive on its barriers
  if (csize > 1) cluster_sync();
}

template <int kBf16, bool kTop, int kWarps, int kSlice, int kMinBlocks>
cudaError_t launch_stream(int cluster, int N, int sms, const uint8_t* z, int64_t ld_bytes,
                          const int32_t* tokens, int V, int ignore_index, int top_k, float inv_t,
                          float* logprob, float* entropy, float* lse, float* top_lp,
                          int32_t* top_id, int32_t* status, int64_t timeout_ns,
                          cudaStream_t stream) {
  auto kern = logprob_stream_kernel<kBf16, kTop, kWarps, kSlice, kMinBlocks>;
  constexpr int smem = 2 * kSlice;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  int clusters = sms * kMinBlocks / cluster;
  if (clusters < 1) clusters = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((kTop ? kWarps + 3 : kWarps + 2) * 32, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (N < clusters) {
    clusters = N;
  } else if (cluster > 1) {
    // persistent: no more clusters than can be resident at once (asked once per size)
    static std::atomic<int> resident[kMaxRowCluster + 1];
    int active = resident[cluster].load(std::memory_order_relaxed);
    if (active == 0) {
      cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster), 1, 1);
      if (cudaOccupancyMaxActiveClusters(&active, kern, &cfg) != cudaSuccess || active < 1)
        active = clusters;
      resident[cluster].store(active, std::memory_order_relaxed);
    }
    if (active < clusters) clusters = active;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, z, ld_bytes, tokens, N, V, ignore_index, top_k, inv_t,
                            logprob, entropy, lse, top_lp, top_id, status,
                            static_cast<uint64_t>(timeout_ns));
}

// dZ: 16-byte vectors where the row of dZ starts at the same offset from a 16-byte
// boundary as the row of Z, single elements otherwise. A -inf logit gets 0.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;   // vectors per thread

template <int kBf16>
__global__ void __launch_bounds__(kGradThreads, 6)
    logprob_grad_kernel(const uint8_t* z, int64_t ld_bytes,   // may alias g (in place)
                        const int32_t* __restrict__ tokens, int N, int V, int ignore_index,
                        float inv_t, const float* __restrict__ logprob,
                        const float* __restrict__ entropy, const float* __restrict__ lse,
                        const float* __restrict__ dlogprob, const float* __restrict__ dentropy,
                        const float* __restrict__ dlse, uint8_t* g, int64_t gld_bytes) {
  using L = Logit<kBf16>;
  constexpr int E = L::E;
  constexpr int kChunk = kGradThreads * kGradVecs;
  const int tid = threadIdx.x;
  for (int row = blockIdx.y; row < N; row += gridDim.y) {
    const uint8_t* zr = z + static_cast<int64_t>(row) * ld_bytes;
    uint8_t* gr = g + static_cast<int64_t>(row) * gld_bytes;
    const int y = tokens != nullptr ? tokens[row] : ignore_index;
    const int yt = (y == ignore_index || y < 0 || y >= V) ? -1 : y;
    const RowCoef k = row_coef(lse[row], entropy != nullptr ? entropy[row] : 0.f,
                               logprob != nullptr ? logprob[row] : 0.f,
                               dlogprob != nullptr ? dlogprob[row] : 0.f,
                               dentropy != nullptr ? dentropy[row] : 0.f,
                               dlse != nullptr ? dlse[row] : 0.f, yt >= 0, inv_t);
    auto entry = [&](float x) {   // off the token
      const float lp = fmaxf(fmaf(x, inv_t, -k.lse), -1.0e4f);
      const float p = exp2_approx(lp * kLog2e);
      return p * fmaf(-k.B, lp + k.entropy, k.A);
    };
    const bool vectors = ((reinterpret_cast<uintptr_t>(zr) ^ reinterpret_cast<uintptr_t>(gr)) & 15u) == 0;
    const int head = vectors ? row_head<kBf16>(zr, V) : V;
    const int nvec = (V - head) / E;
    const uint8_t* zv = zr + static_cast<int64_t>(head) * L::kBytes;
    uint8_t* gv = gr + static_cast<int64_t>(head) * L::kBytes;
    const int v0 = blockIdx.x * kChunk + tid;
    uint4 w[kGradVecs];
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u)
      if (v0 + u * kGradThreads < nvec)
        w[u] = __ldcs(reinterpret_cast<const uint4*>(zv) + v0 + u * kGradThreads);
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
      const int v = v0 + u * kGradThreads;
      if (v < nvec) {
        float x[E];
        L::widen(w[u], x);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = entry(x[e]);
        const int at = yt - (head + v * E);
        if (static_cast<unsigned>(at) < static_cast<unsigned>(E)) {   // the token's vector
          const float target = target_entry(k.target, element_of<kBf16>(w[u], at));
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (e == at) x[e] = target;
        }
        __stcs(reinterpret_cast<uint4*>(gv) + v, L::narrow(x));
      }
    }
    // single elements: those before the vectors (all of the row without them) and after
    const int tail = head + nvec * E;
    const int singles = head + (V - tail);
    for (int i = blockIdx.x * kGradThreads + tid; i < singles; i += gridDim.x * kGradThreads) {
      const int id = i < head ? i : tail + i - head;
      const float x = L::load1(zr + static_cast<int64_t>(id) * L::kBytes);
      L::store1(gr + static_cast<int64_t>(id) * L::kBytes, id == yt ? target_entry(k.target, x) : entry(x));
    }
  }
}

}  // namespace

cudaError_t launch_logprob_rows(int bf16, const void* z, int64_t ld_bytes, const int32_t* tokens,
                                int N, int V, int ignore_index, int top_k, float inv_t,
                                float* logprob, float* entropy, float* lse, float* top_lp,
                                int32_t* top_id, int32_t* status, int sms, int64_t timeout_ns,
                                cudaStream_t stream) {
  const uint8_t* zp = static_cast<const uint8_t*>(z);
  const int64_t row_bytes = static_cast<int64_t>(V) * (bf16 ? 2 : 4);
  // Slices: rows of up to 20 KB whole in CTAs of 4 warps for the passes (four per SM), others in
  // slices of at most 49 KB in CTAs of 8 (two per SM), or, when eight of those do not hold the
  // row, 104 KB in CTAs of 16 (one); and two more warps each, three with a ranking. In us without
  // and with 5 alternatives, the kernel taken / the next one up:
  //   a warp per row to 8 KB : 16384 x 2000 bf16 17.4, 26.0 / 37.0, 55.0; 8192 x 4000 19.8, 29.4 /
  //                            23.7, 31.9
  //   20 KB, four per SM     : 4096 x 8000 bf16 18.6, 23.5 / 21.6, 31.6
  //   49 KB, two per SM      : 8192 x 128256 bf16 370, 494 / 390, 502; 4096 x 20000 35, 44 / 45, 69
  //   104 KB, one per SM     : 512 x 180000 fp32 72, 91 / 125, 128 (rows read twice)
  constexpr int kWarpRow = 8 << 10, kSmall = 20 << 10, kTwo = 49 << 10, kOne = 104 << 10;
  auto cluster_for = [&](int64_t slice) {
    // whole 16-byte vectors per CTA: leave one vector for the rounding up
    return static_cast<int>((row_bytes + slice - 17) / (slice - 16));
  };
  auto go = [&](auto b, auto t) {
    using std::integral_constant;
    auto warp_rows = [&](auto nv) {
      logprob_warp_kernel<b(), t(), nv()>
          <<<(N + kWarpRowWarps - 1) / kWarpRowWarps, kWarpRowWarps * 32, 0, stream>>>(
              zp, ld_bytes, tokens, N, V, ignore_index, top_k, inv_t, logprob, entropy, lse,
              top_lp, top_id, status);
      return cudaGetLastError();
    };
    if (row_bytes <= kWarpRow / 4) return warp_rows(integral_constant<int, 4>{});
    if (row_bytes <= kWarpRow / 2) return warp_rows(integral_constant<int, 8>{});
    if (row_bytes <= kWarpRow) return warp_rows(integral_constant<int, 16>{});
    auto run = [&](auto warps, auto slice, auto blocks, int cluster) {
      return launch_stream<b(), t(), warps(), slice(), blocks()>(
          cluster, N, sms, zp, ld_bytes, tokens, V, ignore_index, top_k, inv_t, logprob, entropy,
          lse, top_lp, top_id, status, timeout_ns, stream);
    };
    int cl = cluster_for(kSmall);
    if (cl <= 1)
      return run(integral_constant<int, 4>{}, integral_constant<int, kSmall>{}, integral_constant<int, 4>{}, 1);
    cl = cluster_for(kTwo);
    // few rows of several CTAs: more for each, down to 8 KB, until half of the SMs have one. One
    // row of 128256 fp32 logits 5.6 us on 8 CTAs, 6.5 on 6; 16 rows of bf16 6.2 on 8, 5.9 on 6;
    // one row of 24 KB 4.7 on 3 against 3.7 on one.
    int spread = cl > 1 ? sms / (2 * N) : 1;
    const int most = static_cast<int>((row_bytes + (8 << 10) - 1) / (8 << 10));
    spread = spread < most ? spread : most;
    spread = spread < kMaxRowCluster ? spread : kMaxRowCluster;
    if (cl <= kMaxRowCluster)
      return run(integral_constant<int, 8>{}, integral_constant<int, kTwo>{}, integral_constant<int, 2>{},
                 cl > spread ? cl : spread);
    cl = cluster_for(kOne);
    if (cl <= kMaxRowCluster)
      return run(integral_constant<int, 16>{}, integral_constant<int, kOne>{}, integral_constant<int, 1>{},
                 cl > spread ? cl : spread);
    const int grid = N < sms * 4 ? N : sms * 4;
    logprob_rows_kernel<b(), t()><<<grid, kRowThreads, 0, stream>>>(
        zp, ld_bytes, tokens, N, V, ignore_index, top_k, inv_t, logprob, entropy, lse, top_lp,
        top_id, status);
    return cudaGetLastError();
  };
  if (bf16) return top_k ? go(std::integral_constant<int, 1>{}, std::true_type{})
                         : go(std::integral_constant<int, 1>{}, std::false_type{});
  return top_k ? go(std::integral_constant<int, 0>{}, std::true_type{})
               : go(std::integral_constant<int, 0>{}, std::false_type{});
}

cudaError_t launch_logprob_grad(int bf16, const void* z, int64_t ld_bytes, const int32_t* tokens,
                                int N, int V, int ignore_index, float inv_t, const float* logprob,
                                const float* entropy, const float* lse, const float* dlogprob,
                                const float* dentropy, const float* dlse, void* g,
                                int64_t gld_bytes, cudaStream_t stream) {
  const int E = bf16 ? 8 : 4;
  const int chunk = kGradThreads * kGradVecs * E;
  const dim3 grid(static_cast<unsigned>((V + chunk - 1) / chunk),
                  static_cast<unsigned>(N < 65535 ? N : 65535));
  auto go = [&](auto kern) {
    kern<<<grid, kGradThreads, 0, stream>>>(static_cast<const uint8_t*>(z), ld_bytes, tokens, N, V,
                                            ignore_index, inv_t, logprob, entropy, lse, dlogprob,
                                            dentropy, dlse, static_cast<uint8_t*>(g), gld_bytes);
    return cudaGetLastError();
  };
  return bf16 ? go(logprob_grad_kernel<1>) : go(logprob_grad_kernel<0>);
}

}  // namespace flce
