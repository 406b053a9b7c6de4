// Log probabilities of given tokens over a logits matrix Z [N, V] (fp32 or bf16), with
// each row's entropy and most likely ids, and their gradient in the logits.
//
// Forward, one row per CTA: pass 1 takes the maximum, pass 2 sums 2^d and 2^d d against
// it (flce_rowstat.cuh) and collects the candidates of the ranking. Any element of the
// top k is at least as large as the k-th largest of 32 maxima over disjoint groups of
// threads, since those k groups hold k elements that large; pass 1 gives those maxima,
// so pass 2 only keeps the elements that reach that threshold, about 2 k of them on
// logits without many equal values. One warp sorts them. A row where too many reach it
// (most of its logits equal) is ranked by k passes instead, each the largest key below
// the one before.
//
// Backward, elementwise: every entry of dZ from its logit and five numbers of its row.
//
// Rows may start at any element: the elements before the first 16-byte boundary and
// after the last one are read singly.
#include <cmath>
#include <cstdint>

#include "flce_internal.h"
#include "flce_rowstat.cuh"
#include "flce_topk.cuh"

namespace flce {

namespace {

constexpr int kRowThreads = 512;
constexpr int kCandidates = 1024;

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
      // the difference first: x c alone overflows for a mask of the type's lowest value
      const float d = fmaxf((x - M) * c, kMinExponent);
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

// dZ: 16-byte vectors where the row of dZ starts at the same offset from a 16-byte
// boundary as the row of Z, single elements otherwise. A -inf logit gets 0.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;   // vectors per thread

template <int kBf16>
__global__ void __launch_bounds__(kGradThreads)
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
    auto entry = [&](float x, int id) {
      if (id == yt) return k.target;
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
        for (int e = 0; e < E; ++e) x[e] = entry(x[e], head + v * E + e);
        __stcs(reinterpret_cast<uint4*>(gv) + v, L::narrow(x));
      }
    }
    // single elements: those before the vectors (all of the row without them) and after
    const int tail = head + nvec * E;
    const int singles = head + (V - tail);
    for (int i = blockIdx.x * kGradThreads + tid; i < singles; i += gridDim.x * kGradThreads) {
      const int id = i < head ? i : tail + i - head;
      const float x = L::load1(zr + static_cast<int64_t>(id) * L::kBytes);
      L::store1(gr + static_cast<int64_t>(id) * L::kBytes, entry(x, id));
    }
  }
}

}  // namespace

cudaError_t launch_logprob_rows(int bf16, const void* z, int64_t ld_bytes, const int32_t* tokens,
                                int N, int V, int ignore_index, int top_k, float inv_t,
                                float* logprob, float* entropy, float* lse, float* top_lp,
                                int32_t* top_id, int32_t* status, int sms, cudaStream_t stream) {
  const uint8_t* zp = static_cast<const uint8_t*>(z);
  const int grid = N < sms * 4 ? N : sms * 4;
  auto go = [&](auto kern) {
    kern<<<grid, kRowThreads, 0, stream>>>(zp, ld_bytes, tokens, N, V, ignore_index, top_k, inv_t,
                                           logprob, entropy, lse, top_lp, top_id, status);
    return cudaGetLastError();
  };
  if (bf16) return top_k ? go(logprob_rows_kernel<1, true>) : go(logprob_rows_kernel<1, false>);
  return top_k ? go(logprob_rows_kernel<0, true>) : go(logprob_rows_kernel<0, false>);
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
