// Persistent, warp-specialised tcgen05 GEMM for sm_103a with six fused
// epilogues. Every product of fused linear cross-entropy runs through it:
//
//   LSE  : Z = H W^T tile by tile, accumulated in TMEM; the epilogue keeps a
//          per-token running max and sum of exponentials (the target's own term
//          left out) across the vocabulary tiles of a work unit and extracts the
//          target logit ("Liger Kernel: Fused Triton Kernels for LLM Training",
//          The Architecture, 1. steps 2-5: in-SRAM tile product, online
//          LogSumExp, immediate target extraction, no logits written).
//   GRAD : Z recomputed tile by tile; the epilogue forms
//          G = (exp(z - lse) - [v = y]) * scale in bf16, as exp(z - max) * scale /
//          sum off the target and -scale * (1 - p) at it, and writes one chunk of
//          G, stored chunk-major (same page, 2. In-Kernel Gradient Computation:
//          recompute the tile logits from the saved LSE, derive dL/dz in the kernel).
//   LOGP : as LSE, with the sum that the entropy needs (log probabilities of given
//          tokens); LOGP_TOP also ranks each token's largest logits on the fly.
//   LOGP_GRAD : as GRAD, with G = p (A - B (log p + entropy)) from per-token upstream
//          gradients, and the token's own entry given.
//   F32  : plain product whose tile is stored as fp32, added to fp32 already in
//          memory, or stored as bf16 — used for dW = G^T H and dH = G W (same
//          page, 2.).
//
// CTA layout (192 threads, one CTA per SM). kCta = 1: each CTA computes a
// 128 x 256 tile. kCta = 2: a cluster pair computes a 256 x 256 tile with
// tcgen05 cta_group::2 MMAs; each CTA holds its 128 rows of A and 128 of the 256
// rows of B, and its own 128 x 256 fp32 accumulator rows in TMEM.
//   warp 0     : TMA producer (each CTA; all lanes wait, one elected lane issues)
//                — streams the CTA's A rows and B half, K-slice by K-slice, into a
//                ring of shared-memory stages; the copies of both CTAs complete on
//                the even CTA's stage barrier. With k_serpentine, every second tile
//                of a pair walks K from the end, so that it starts on the K slices
//                the tiles before it read last, which are the ones still in L2.
//   warp 1     : TMEM allocator (both CTAs) and MMA issuer (the even CTA's warp:
//                all lanes wait on the barriers, one elected lane issues the
//                tcgen05.mma M x 256 x 16 steps into one of two TMEM accumulators
//                and the commits).
//   warps 2..5 : epilogue — warp w reads TMEM lanes 32*(w%4) .. +31, so each
//                thread owns one output row of its CTA's 128 rows; tiles that
//                leave the SM go through per-warp 32 x 32 staging boxes in shared
//                memory and TMA stores (or reduce-adds).
// Every wait is bounded (see mbar_wait_bounded); on a timeout the CTA records
// FLCE_ERR_TIMEOUT, the producer drains the copies it issued, the MMA warp
// drains its MMAs, and both CTAs free TMEM and exit.
#pragma once

#include <cmath>
#include <cstdint>

#include "flce_gemm_params.h"
#include "flce_rowstat.cuh"
#include "flce_topk.cuh"
#include "ptx.cuh"

namespace flce {

// Units are ordered in groups of group_m row tiles; inside a group the column
// index (EPI_LSE: the vocabulary range) is the outer loop, so the tiles running at
// the same time share both their A row blocks and their B column blocks.
// Returns the column index (EPI_LSE: the vocabulary range) of unit u.
template <int kEpi>
__device__ __forceinline__ int unit_tiles(const GemmParams& p, int u, int& m_blk, int& n_begin,
                                          int& n_end) {
  const int n_units_per_row = epi_sums_rows(kEpi) ? p.splits : p.n_blocks;
  const int per_group = p.group_m * n_units_per_row;
  const int g = u / per_group;
  const int first_m = g * p.group_m;
  const int gm = min(p.m_blocks - first_m, p.group_m);
  const int r = u - g * per_group;
  const int col = r / gm;
  m_blk = first_m + (r - col * gm);
  if constexpr (epi_sums_rows(kEpi)) {
    n_begin = static_cast<int>((static_cast<int64_t>(col) * p.n_blocks) / p.splits);
    n_end = static_cast<int>((static_cast<int64_t>(col + 1) * p.n_blocks) / p.splits);
  } else {
    n_begin = col;
    n_end = col + 1;
  }
  return col;
}

__device__ __forceinline__ void record_status(int32_t* status, int code) {
  if (status != nullptr) atomicCAS(reinterpret_cast<int*>(status), 0, code);
}

// ---- epilogue bodies ---------------------------------------------------------------

struct LseState {
  float m;   // running max of z (the target's logit included)
  float s;   // running sum of exp(z - m) over every column but the target's
  float zt;  // target logit
  bool found;
};

// One 32-column chunk of the logits tile for this thread's row. The target's own
// term is left out of the sum (the merge adds it back), so that 1 - p of the
// target, the sum of the other terms over the whole sum, is known without a
// difference of nearly equal numbers.
__device__ __forceinline__ void lse_chunk(const float (&v)[32], int col_local, int n_valid,
                                          int rel_target, LseState& st) {
  float x[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) x[k] = v[k];
  if (col_local + 32 > n_valid) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (col_local + k >= n_valid) x[k] = -INFINITY;
  }
  float c0 = fmaxf(x[0], x[1]), c1 = fmaxf(x[2], x[3]);
#pragma unroll
  for (int k = 4; k < 32; k += 4) {
    c0 = fmaxf(c0, fmaxf(x[k], x[k + 1]));
    c1 = fmaxf(c1, fmaxf(x[k + 2], x[k + 3]));
  }
  const float mn = fmaxf(st.m, fmaxf(c0, c1));
  if (static_cast<unsigned>(rel_target) < 32u) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (k == rel_target) {
        st.zt = v[k];
        x[k] = -INFINITY;   // in the max above, not in the sum below
      }
    st.found = true;
  }
  if (mn == -INFINITY) return;
  const float ms = mn * kLog2e;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    s0 += ex2_approx(fmaf(x[k + 0], kLog2e, -ms));
    s1 += ex2_approx(fmaf(x[k + 1], kLog2e, -ms));
    s2 += ex2_approx(fmaf(x[k + 2], kLog2e, -ms));
    s3 += ex2_approx(fmaf(x[k + 3], kLog2e, -ms));
  }
  st.s = st.s * ex2_approx((st.m - mn) * kLog2e) + ((s0 + s1) + (s2 + s3));
  st.m = mn;
}

// A token's ranking within its vocabulary range. The thread that owns the row appends the
// logits that beat its bound, the smallest of its top_k so far, to kBeat entries in shared
// memory; when some row of the warp could not take another four columns, every thread cuts
// its entries down to its top_k: a sorting network over their values gives the top_k-th, and
// one pass keeps what reaches it. All 32 rows of the warp do that at once, about 1000
// instructions for the warp, ln(range / top_k) or so times per range and token.
// Measured at 8192 x 4096 x 128256 (4.28 ms without alternatives) with 5, 20 and 32: 4.33, 4.46,
// 4.77 ms; with a bound per range alone, below, 4.37, 4.72, 10.0. Earlier, against 4.75 ms without,
// with 20: inserting each candidate into a sorted list by its own thread 37.4 ms, joining buffers
// and lists row by row with a key per lane 7.6. Looking every eight columns leaves one entry of
// room with 32: 2048 tokens 4.99 ms against 1.55; every two took 1% more with 16 or fewer.
//
// An entry is the logit and its column within the range (16 bits: the ranges are planned to
// have at most 65536 columns), entry e of the CTA's 128 rows contiguous, so that the threads
// of a warp never conflict.
constexpr int kBeat = 40;

// Compare-exchange, the larger value first.
__device__ __forceinline__ void order_desc(float& a, float& b) {
  const float hi = fmaxf(a, b);
  b = fminf(a, b);
  a = hi;
}

// Steps kJ, kJ / 2, ... 1 of a bitonic network over x[0, 32): blocks of kSize in alternating
// order (kSize = 32: descending).
template <int kSize, int kJ>
__device__ __forceinline__ void bitonic_steps(float (&x)[kBeat]) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if ((e & kJ) == 0) {
      if ((e & kSize) == 0) order_desc(x[e], x[e | kJ]);
      else order_desc(x[e | kJ], x[e]);
    }
  if constexpr (kJ > 1) bitonic_steps<kSize, kJ / 2>(x);
}
template <int kSize>
__device__ __forceinline__ void bitonic_sort(float (&x)[kBeat]) {
  if constexpr (kSize > 2) bitonic_sort<kSize / 2>(x);
  bitonic_steps<kSize, kSize / 2>(x);
}
// One step of odd-even transposition over x[32, 40), smaller values first.
template <int kStep>
__device__ __forceinline__ void transpose_steps(float (&x)[kBeat]) {
#pragma unroll
  for (int e = kStep & 1; e + 1 < 8; e += 2) order_desc(x[32 + e + 1], x[32 + e]);
  if constexpr (kStep < 7) transpose_steps<kStep + 1>(x);
}

struct RankCut {
  float bound;
  int count;
};

// A token's ranges, in whatever order they run, tell each other their bounds: the top_k-th of
// some of the row is no more than that of the whole, so logits below it need not be kept.
// Those equal to it must, as they may have lower ids: the bound taken over is a little less.
// (Which entries are kept on the way depends on the order, the top_k of them all do not.)
__device__ __forceinline__ float just_below(uint32_t bits) {
  const float v = bits == 0 ? -INFINITY : ordered_value(bits);
  return fabsf(v) < INFINITY ? v - (fabsf(v) * 2.4e-7f + 1e-37f) : -INFINITY;
}
__device__ __forceinline__ uint32_t ld_relaxed_u32(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Cuts a row's entries down to the top_k largest, in the order they came (ascending ids);
// the new bound is the smallest of them. `values` and `columns` are the shared-memory
// addresses of the row's entries. Not inlined: its 1000 instructions four times over in
// the loop over the tile's columns evict the loop from the instruction cache.
static __device__ __noinline__ RankCut rank_cut(uint32_t values, uint32_t columns, int count, int top_k) {
  if (count < top_k) return RankCut{-INFINITY, count};
  float x[kBeat];
#pragma unroll
  for (int e = 0; e < kBeat; ++e) {
    x[e] = -INFINITY;
    if (e < count) x[e] = ld_shared_f32(values + e * (BM * 4));
  }
  bitonic_sort<32>(x);
  transpose_steps<0>(x);
  // the 32 largest of both: the maxima of the smallest 8 of one with the other are bitonic
#pragma unroll
  for (int e = 0; e < 8; ++e) x[24 + e] = fmaxf(x[24 + e], x[32 + e]);
  bitonic_steps<32, 16>(x);
  float bound = x[0];
  int equal = 1;   // entries at the bound that stay
#pragma unroll
  for (int e = 1; e < 32; ++e)
    if (e < top_k) {
      equal = x[e] == bound ? equal + 1 : 1;
      bound = x[e];
    }
  int kept = 0;
#pragma unroll 8
  for (int e = 0; e < kBeat; ++e) {
    const float v = ld_shared_f32(values + e * (BM * 4));
    const uint32_t c = ld_shared_u16(columns + e * (BM * 2));
    if (e < count && (v > bound || (v == bound && equal > 0))) {
      if (v == bound) --equal;
      st_shared_f32(values + kept * (BM * 4), v);
      st_shared_u16(columns + kept * (BM * 2), c);
      ++kept;
    }
  }
  return RankCut{bound, kept};
}

// Running row state of the log-probability epilogue. The logits are raw: c = log2(e) /
// temperature is applied in the exponent.
struct LogpState {
  RowPart p;   // running max, sum 2^d, sum 2^d d (flce_rowstat.cuh), the token's term left out
  float zt;
  bool found;
};

// What takes the token's place in the sums: 2^d = 0 and d finite, so that 2^d d is 0 too
// (temperatures are at least 1e-6).
constexpr float kNoLogit = -1.0e30f;

// lse_chunk with the entropy's sum; columns past the product count as logits of -inf. Returns
// the chunk's largest logit.
//
// The exponents are not floored one by one (8192 x 4096 x 128256 with 5 alternatives: 5.02 ms
// against 4.75). A logit of -inf, an id that cannot come, then makes 2^d d = 0 * -inf a NaN, which
// sends the warp through the chunk again with the floor.
__device__ __forceinline__ float logp_chunk(const float (&v)[32], int col_local, int n_valid,
                                            int rel_target, float c, LogpState& st) {
  float x[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) x[k] = v[k];
  if (col_local + 32 > n_valid) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (col_local + k >= n_valid) x[k] = -INFINITY;
  }
  float c0 = max_nan(x[0], x[1]), c1 = max_nan(x[2], x[3]);
#pragma unroll
  for (int k = 4; k < 32; k += 4) {
    c0 = max_nan(c0, max_nan(x[k], x[k + 1]));
    c1 = max_nan(c1, max_nan(x[k + 2], x[k + 3]));
  }
  const float cm = max_nan(c0, c1);
  const float mn = max_nan(st.p.m, cm);
  if (static_cast<unsigned>(rel_target) < 32u) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (k == rel_target) {
        st.zt = v[k];
        x[k] = kNoLogit;   // in the max above, not in the sums below
      }
    st.found = true;
  }
  float s0, s1, t0, t1;
  auto sums = [&](auto exponent) {
    s0 = s1 = t0 = t1 = 0.f;
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const float d0 = exponent(x[k]), d1 = exponent(x[k + 1]);
      const float e0 = exp2_approx(d0), e1 = exp2_approx(d1);
      s0 += e0;
      s1 += e1;
      t0 = fmaf(e0, d0, t0);
      t1 = fmaf(e1, d1, t1);
    }
  };
  const float ref = row_ref(mn, c);
  float dm = 0.f;
  bool floored = !__all_sync(0xffffffffu, has_ref(mn, c));   // or very low temperatures
  if (!floored) {
    sums([&](float z) { return fmaf(z, c, -ref); });
    dm = fmaxf(row_ref(st.p.m, c) - ref, kMinExponent);
    const float t = t0 + t1;
    floored = __any_sync(0xffffffffu, t != t);
  }
  if (floored) {
    // (the token's place against a maximum of -inf, or below its stand-in, would count)
    sums([&](float z) { return z == kNoLogit ? kMinExponent : row_exponent(z, mn, c); });
    dm = row_shift(st.p.m, mn, c);
  }
  const float f = exp2_approx(dm);
  st.p.t = fmaf(fmaf(st.p.s, dm, st.p.t), f, t0 + t1);
  st.p.s = fmaf(st.p.s, f, s0 + s1);
  st.p.m = mn;
  return cm;
}

// G for one 32-column chunk of the log-probability gradient: l = log p,
// p (A - B (l + entropy)) off the token and `target` at it, 0 past n_valid.
__device__ __forceinline__ void logp_grad_chunk(const float (&v)[32], int col_local, int n_valid,
                                                int rel_target, float inv_t, const float4& k4,
                                                float target, float (&g)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float l = fmaxf(fmaf(v[k], inv_t, -k4.x), -1.0e4f);   // p l of a logit of -inf is 0
    g[k] = ex2_approx(l * kLog2e) * fmaf(-k4.z, l + k4.w, k4.y);
  }
  if (static_cast<unsigned>(rel_target) < 32u) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (k == rel_target) g[k] = target_entry(target, v[k]);
  }
  if (col_local + 32 > n_valid) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (col_local + k >= n_valid) g[k] = 0.f;
  }
}

// Epilogue staging. Each epilogue warp writes its 32 rows x 32 columns into a
// shared-memory box in the layout the output map's swizzle expects, then one lane
// hands the box to a TMA store: the global writes leave the SM as whole lines
// instead of one 16-byte piece of 32 different rows per store instruction.
//   fp32 box: rows of 128 bytes, 128-byte swizzle: 16-byte chunk q of row r sits
//             at chunk q ^ (r % 8);
//   bf16 box: rows of 64 bytes, 64-byte swizzle: chunk q of row r at q ^ ((r / 2) % 4).
__device__ __forceinline__ void stage_f32_row(uint32_t box, int r, const float (&v)[32]) {
  const uint32_t row = box + static_cast<uint32_t>(r) * 128u;
#pragma unroll
  for (int q = 0; q < 8; ++q)
    st_shared_v4(row + ((static_cast<uint32_t>(q ^ (r & 7))) << 4), __float_as_uint(v[4 * q]),
                 __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                 __float_as_uint(v[4 * q + 3]));
}

__device__ __forceinline__ void stage_bf16_row(uint32_t box, int r, const float (&v)[32]) {
  const uint32_t row = box + static_cast<uint32_t>(r) * 64u;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    st_shared_v4(row + ((static_cast<uint32_t>(q ^ ((r >> 1) & 3))) << 4),
                 pack_bf16x2(v[8 * q + 0], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                 pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
}

// G for one 32-column chunk: (exp(z - zmax) * a - [v = y] * sc, 0 past n_valid,
// with a = sc / sum exp(z - zmax) (or zmax = lse and a = sc). The exponent's
// difference is taken first, exact when z is close to zmax. The target entry is
// -sc * q with q = 1 - p as the merge formed it, when q >= 0 is given; else
// (a vocabulary shard, which has only lse) exp(z - lse) * sc - sc.
__device__ __forceinline__ void grad_chunk(const float (&v)[32], int col_local, int n_valid,
                                           int rel_target, float zmax, float a, float sc,
                                           float q, float (&g)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k) g[k] = ex2_approx((v[k] - zmax) * kLog2e) * a;
  if (static_cast<unsigned>(rel_target) < 32u) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (k == rel_target) g[k] = q >= 0.f ? -sc * q : g[k] - sc;
  }
  if (col_local + 32 > n_valid) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (col_local + k >= n_valid) g[k] = 0.f;
  }
}

// ---- the kernel --------------------------------------------------------------------

// kFp8 = 1: A and B are E4M3 bytes (K-major only), 128 of them per 128-byte
// stage row, multiplied with tcgen05 kind::f8f6f4; the epilogue scales z by
// the product of the two device scales. The shared-memory image of a stage is
// the same as for bf16.
// kWide = 1: 256 x 512 tiles (TileCfg): each CTA stages two 128-row halves of B
// per K block, the MMA thread issues one N = 256 MMA per half into columns
// [256 h, 256 h + 256) of the single accumulator, and tile column c is product
// column n_blk * 512 + c.
// kProducts = 2: one launch computes two independent products of the same tile
// shape and epilogue, g0's units first, then g1's (the dH and dW products of a
// vocabulary chunk, which both only read G). Units are dealt to the pairs in that
// fixed order, each unit taking its maps and parameters from its own product, so
// every output element still has one writer per launch.
template <int kEpi, int kCta, int kFp8 = 0, int kWide = 0, int kProducts = 1>
__global__ void __launch_bounds__(kThreads, 1)
    flce_gemm_kernel(const __grid_constant__ GemmArgs g0, const __grid_constant__ GemmArgs g1) {
  using Cfg = TileCfg<kCta, kWide>;
  static_assert(kWide == 0 || kEpi == EPI_F32, "wide tiles carry the fp32 epilogue only");
  static_assert(kProducts == 1 || kEpi == EPI_F32, "two products per launch: fp32 epilogue only");
  constexpr int kStages = Cfg::kStages;
  constexpr int kSub = Cfg::kSub;
  // settings shared by every unit of the launch come from the first product
  const GemmParams& p0 = g0.p;
  const int units0 = p0.num_units;
  const int total_units = units0 + (kProducts == 2 ? g1.p.num_units : 0);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kRingBytes + 8 * Cfg::kStgBytes);
  // bars: full[kStages] | empty[kStages] | tfull[2] | tempty[2] | drain
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = (kCta == 2) ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x) / kCta;
  const int num_pairs = static_cast<int>(gridDim.x) / kCta;
  const uint32_t stage0 = smem_u32(smem);
  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + kStages + s); };
  auto tfull_bar = [&](int a) { return smem_u32(bars + 2 * kStages + a); };
  auto tempty_bar = [&](int a) { return smem_u32(bars + 2 * kStages + 2 + a); };
  const uint32_t drain_bar = smem_u32(bars + 2 * kStages + 4);
  constexpr bool kCl = kCta == 2;  // waits acquire at cluster scope in pair mode

  if (threadIdx.x == 0) {
    // full[s] of the even CTA counts the copies of both CTAs of a pair (the odd
    // CTA's copies complete on it remotely); the odd CTA's full[s] is unused.
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4 * kCta);  // four epilogue warps per CTA
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&g0.a);
    tma_prefetch_desc(&g0.b);
    if constexpr (!epi_sums_rows(kEpi)) tma_prefetch_desc(&g0.c);
    if constexpr (kProducts == 2) {
      tma_prefetch_desc(&g1.a);
      tma_prefetch_desc(&g1.b);
      tma_prefetch_desc(&g1.c);
    }
  }
  // Barriers of both CTAs are initialised before either CTA touches the other's.
  if constexpr (kCta == 2) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tmem_alloc_cg<kCta>(smem_u32(tmem_holder), kTmemCols);
    tmem_relinquish_cg<kCta>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  const uint64_t tmo = p0.timeout_ns;

  if (warp == 0) {
    // ---------------- TMA producer (each CTA loads its own A rows and B half) -----
    {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued_mask = 0, issued_par = 0;
      bool ok = true;
      const uint64_t pol_a = make_l2_policy(p0.a_hint);
      const uint64_t pol_b = make_l2_policy(p0.b_hint);
      int tile_it = 0;
      for (int u = pair; ok && u < total_units; u += num_pairs) {
        const bool second = kProducts == 2 && u >= units0;
        const GemmArgs& G = second ? g1 : g0;
        const GemmParams& p = G.p;
        const int k_stages = (p.k_blocks + kSub - 1) / kSub;  // ring stages per tile
        int m_blk, n_begin, n_end;
        unit_tiles<kEpi>(p, second ? u - units0 : u, m_blk, n_begin, n_end);
        for (int n_blk = n_begin; ok && n_blk < n_end; ++n_blk, ++tile_it) {
          const bool k_rev = p.k_serpentine && (tile_it & 1);
          for (int kq = 0; kq < k_stages; ++kq) {
            const int ks = k_rev ? k_stages - 1 - kq : kq;   // K block group this stage holds
            const bool empty_ok = mbar_wait_bounded<kCl>(empty_bar(stage), phase ^ 1u, tmo, abort_flag);
            if (!__all_sync(0xffffffffu, empty_ok)) {  // one decision for the whole warp
              ok = false;
              break;
            }
            if (elect_one()) {
            const int nsub = min(kSub, p.k_blocks - ks * kSub);
            const uint32_t fb_local = full_bar(stage);
            if (leader)
              mbar_arrive_expect_tx(fb_local, static_cast<uint32_t>(kCta * nsub) * Cfg::kSubBytes);
            // copies complete on the even CTA's barrier
            const uint32_t fb = (kCta == 2) ? mapa_shared(fb_local, 0) : fb_local;
            const int am = m_blk * Cfg::kTileM + static_cast<int>(rank) * BM;   // A rows
            auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t pol) {
              if constexpr (kCta == 2) tma_load_2d_pair(dst, map, x, y, fb, pol);
              else tma_load_2d_hint(dst, map, x, y, fb, pol);
            };
            auto load3 = [&](uint32_t dst, const CUtensorMap* map, int y, int z, uint64_t pol) {
              if constexpr (kCta == 2) tma_load_3d_pair(dst, map, 0, y, z, fb, pol);
              else tma_load_3d_hint(dst, map, 0, y, z, fb, pol);
            };
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
              if (sub >= nsub) break;
              const int kx = (ks * kSub + sub) * (kFp8 ? 2 * BK : BK);  // elements per 128-byte row
              const uint32_t sa = stage0 + stage * Cfg::kStageBytes + sub * Cfg::kSubBytes;
              const uint32_t sb = sa + Cfg::kABytes;
              if (!p.a_mn_major && p.a_kchunk) {
                load3(sa, &G.a, am + p.a_mn0, (kx + p.a_k0) >> 6, pol_a);
              } else if (!p.a_mn_major) {
                load(sa, &G.a, kx + p.a_k0, am + p.a_mn0, pol_a);
              } else if (p.a_box3) {
                load3(sa, &G.a, kx + p.a_k0, (am + p.a_mn0) >> 6, pol_a);
              } else {
#pragma unroll
                for (int j = 0; j < BM / 64; ++j)
                  load(sa + j * kMnBoxBytes, &G.a, am + 64 * j + p.a_mn0, kx + p.a_k0, pol_a);
              }
#pragma unroll
              for (int h = 0; h < Cfg::kBHalves; ++h) {
                // B rows of this CTA for the MMA of tile columns [256 h, 256 h + 256)
                const int bn = n_blk * Cfg::kTileN + h * BN + static_cast<int>(rank) * Cfg::kBRows;
                const uint32_t sbh = sb + h * Cfg::kBHalfBytes;
                if (!p.b_mn_major) {
                  load(sbh, &G.b, kx + p.b_k0, bn + p.b_mn0, pol_b);
                } else if (p.b_box3) {
                  load3(sbh, &G.b, kx + p.b_k0, (bn + p.b_mn0) >> 6, pol_b);
                } else {
#pragma unroll
                  for (int j = 0; j < Cfg::kBRows / 64; ++j)
                    load(sbh + j * kMnBoxBytes, &G.b, bn + 64 * j + p.b_mn0, kx + p.b_k0, pol_b);
                }
              }
            }
            }
            __syncwarp();
            issued_mask |= 1u << stage;
            issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      if (!ok) {
        if (lane == 0) record_status(p0.status, kStatusTimeout);
        *abort_flag = 1;
      }
      // Drain before the final barrier. The even CTA waits for every stage phase it
      // armed; those phases count the odd CTA's copies too, and in a normal run the
      // odd CTA issues exactly those phases. After an abort the odd CTA may have
      // issued a phase the even CTA never armed, which it cannot observe: it then
      // waits a bounded grace period (far longer than a copy takes) so that its
      // copies land while both CTAs are still resident.
      const volatile int no_abort = 0;
      if (leader) {
        for (int s = 0; s < kStages; ++s)
          if (issued_mask & (1u << s))
            mbar_wait_bounded<kCl>(full_bar(s), (issued_par >> s) & 1u, 1000000000ull, &no_abort);
      } else if (!ok || *abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer (even CTA) ----------------
    if (leader) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      bool issued_any = false;
      int tile_it = 0;
      for (int u = pair; ok && u < total_units; u += num_pairs) {
        const bool second = kProducts == 2 && u >= units0;
        const GemmParams& p = second ? g1.p : g0.p;
        const int k_stages = (p.k_blocks + kSub - 1) / kSub;  // ring stages per tile
        const int k_blocks = p.k_blocks;
        const bool a_mn = p.a_mn_major != 0, b_mn = p.b_mn_major != 0;
        const uint32_t idesc = p.idesc;
        const bool serp = p.k_serpentine != 0;
        int m_blk, n_begin, n_end;
        unit_tiles<kEpi>(p, second ? u - units0 : u, m_blk, n_begin, n_end);
        for (int n_blk = n_begin; ok && n_blk < n_end; ++n_blk, ++tile_it) {
          const bool k_rev = serp && (tile_it & 1);
          // both CTAs' epilogues must have drained this accumulator
          bool got;
          if constexpr (kCta == 2) {
            got = mbar_try_wait_cluster(tempty_bar(acc), acc_phase ^ 1u);
            if (!got) {
              const uint64_t t0 = global_timer_ns();
              while (!(got = mbar_try_wait_cluster(tempty_bar(acc), acc_phase ^ 1u))) {
                if (*abort_flag || global_timer_ns() - t0 > tmo) break;
              }
            }
          } else {
            got = mbar_wait_bounded(tempty_bar(acc), acc_phase ^ 1u, tmo, abort_flag);
          }
          if (!__all_sync(0xffffffffu, got)) {  // one decision for the whole warp
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * Cfg::kTileN);
          for (int kq = 0; kq < k_stages; ++kq) {
            const bool full_ok = mbar_wait_bounded<kCl>(full_bar(stage), phase, tmo, abort_flag);
            if (!__all_sync(0xffffffffu, full_ok)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const int ks = k_rev ? k_stages - 1 - kq : kq;   // as the producer loaded it
            const int nsub = min(kSub, k_blocks - ks * kSub);
            if (elect_one()) {
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
              if (sub >= nsub) break;
              const uint32_t sa = stage0 + stage * Cfg::kStageBytes + sub * Cfg::kSubBytes;
              const uint32_t sb = sa + Cfg::kABytes;
#pragma unroll
              for (int k = 0; k < BK / UK; ++k) {
                const uint64_t da = a_mn ? make_sw128_desc(sa + k * (UK * 128), kMnBoxBytes, 1024)
                                         : make_sw128_desc(sa + k * (UK * 2), 16, 1024);
                const uint32_t accum = (kq | sub | k) != 0 ? 1u : 0u;   // first MMA of the tile overwrites
#pragma unroll
                for (int h = 0; h < Cfg::kBHalves; ++h) {
                  const uint32_t sbh = sb + h * Cfg::kBHalfBytes;
                  const uint64_t db = b_mn ? make_sw128_desc(sbh + k * (UK * 128), kMnBoxBytes, 1024)
                                           : make_sw128_desc(sbh + k * (UK * 2), 16, 1024);
                  const uint32_t dh = d_tmem + static_cast<uint32_t>(h * BN);
                  if constexpr (kFp8) umma_f8_cg<kCta>(dh, da, db, idesc, accum);
                  else umma_bf16_cg<kCta>(dh, da, db, idesc, accum);
                }
              }
            }
            umma_commit_pair<kCta>(empty_bar(stage));  // frees the stage in both CTAs
            }
            __syncwarp();
            issued_any = true;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (elect_one()) umma_commit_pair<kCta>(tfull_bar(acc));
          __syncwarp();
          if (++acc == Cfg::kAccs) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (!ok) {
        if (lane == 0) record_status(p0.status, kStatusTimeout);
        *abort_flag = 1;
      }
      if (issued_any) {
        // Drain: all MMAs of this warp complete before TMEM is freed.
        const volatile int no_abort = 0;
        if (elect_one()) umma_commit_cg<kCta>(drain_bar);   // the lane that issued them
        __syncwarp();
        mbar_wait_bounded(drain_bar, 0, 1000000000ull, &no_abort);
      }
    }
    __syncwarp();
  } else {
    // ---------------- epilogue warps (both CTAs) ----------------
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // row within this CTA's 128 rows
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tempty_leader0 = (kCta == 2) ? mapa_shared(tempty_bar(0), 0) : tempty_bar(0);
    const uint32_t tempty_leader1 = (kCta == 2) ? mapa_shared(tempty_bar(1), 0) : tempty_bar(1);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    float scale_v = 0.f;
    if constexpr (kEpi == EPI_GRAD) scale_v = *p0.scale;
    float acc_scale = 1.f;  // FP8 operands: product of the two per-tensor scales
    if constexpr (kFp8) acc_scale = *p0.acc_scale_h * *p0.acc_scale_w;
    // this warp's two staging boxes, used alternately
    const uint32_t stg = stage0 + Cfg::kRingBytes + static_cast<uint32_t>(quarter) * 2u * Cfg::kStgBytes;
    uint32_t nbox = 0;
    int stop_u = 0, stop_n = 0;   // the tile that did not come
    for (int u = pair; ok && u < total_units; u += num_pairs) {
      const bool second = kProducts == 2 && u >= units0;
      const GemmArgs& G = second ? g1 : g0;
      const GemmParams& p = G.p;
      int m_blk, n_begin, n_end;
      const int col_unit = unit_tiles<kEpi>(p, second ? u - units0 : u, m_blk, n_begin, n_end);
      const int prow = m_blk * Cfg::kTileM + static_cast<int>(rank) * BM + row;  // product row
      const bool row_ok = prow < p.m_valid;
      int y = -1;
      if constexpr (kEpi != EPI_F32) {
        // the log-probability epilogues may run without tokens
        if (row_ok && (kEpi == EPI_LSE || kEpi == EPI_GRAD || p.labels != nullptr)) {
          const int lab = p.labels[p.row_base + prow];
          y = (lab == p.ignore_index) ? -1 : lab;
        }
      }
      LseState st{-INFINITY, 0.f, 0.f, false};
      // Rows past the product (or of another token block) take zmax = +inf, so
      // their G is exactly 0 whatever logits the tile holds for them.
      float zmax = INFINITY, a = 0.f, sc = 0.f, q = -1.f;
      LogpState lst{{-INFINITY, 0.f, 0.f}, 0.f, false};
      // the ranking's entries are in the staging boxes' 32 KB, which this epilogue does not
      // use otherwise
      const uint32_t rank_values = stage0 + Cfg::kRingBytes + static_cast<uint32_t>(row) * 4u;
      const uint32_t rank_columns =
          stage0 + Cfg::kRingBytes + kBeat * BM * 4u + static_cast<uint32_t>(row) * 2u;
      // -inf until there are top_k entries, +inf for a row that does not exist
      RankCut ranking{row_ok ? -INFINITY : INFINITY, 0};
      uint32_t* const bound_at = p.bounds + prow;
      uint32_t shared_bound = 0;
      if (kEpi == EPI_LOGP_TOP && row_ok) shared_bound = ld_relaxed_u32(bound_at);
      // Rows past the product: log p = -3e38, so p and G are 0.
      float4 k4 = make_float4(3.0e38f, 0.f, 0.f, 0.f);
      float target = 0.f;
      if constexpr (kEpi == EPI_LOGP_GRAD) {
        if (row_ok) {
          k4 = p.coef[p.row_base + prow];
          target = p.target[p.row_base + prow];
        }
      }
      if constexpr (kEpi == EPI_GRAD) {
        if (row_ok) {
          sc = (y >= 0) ? scale_v : 0.f;
          if (p.gstat != nullptr) {
            const float4 gs = p.gstat[p.row_base + prow];
            zmax = gs.x;
            a = sc * gs.y;
            q = gs.z;
          } else {
            zmax = p.lse[p.row_base + prow];
            a = sc;
          }
        }
      }
      for (int n_blk = n_begin; n_blk < n_end; ++n_blk) {
        int got = 0;
        if (lane == 0) {
          if constexpr (kCta == 2) {
            got = mbar_try_wait_cluster(tfull_bar(acc), acc_phase);
            if (!got) {
              const uint64_t t0 = global_timer_ns();
              while (!(got = mbar_try_wait_cluster(tfull_bar(acc), acc_phase))) {
                if (*abort_flag || global_timer_ns() - t0 > tmo) break;
              }
            }
          } else {
            got = mbar_wait_bounded(tfull_bar(acc), acc_phase, tmo, abort_flag) ? 1 : 0;
          }
        }
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          ok = false;
          stop_u = u;
          stop_n = n_blk;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + lane_addr + static_cast<uint32_t>(acc * Cfg::kTileN);
        if constexpr (kEpi == EPI_LOGP_TOP) {
          if (row_ok) {   // what the tile before asked for
            ranking.bound = fmaxf(ranking.bound, just_below(shared_bound));
            shared_bound = ld_relaxed_u32(bound_at);
          }
        }
#pragma unroll 1
        for (int c = 0; c < Cfg::kTileN / 32; ++c) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + c * 32, r);
          tmem_wait_ld();
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
          if constexpr (kFp8) {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] *= acc_scale;
          }
          const int col = n_blk * Cfg::kTileN + c * 32;  // product column
          if constexpr (kEpi == EPI_LSE) {
            lse_chunk(v, col, p.n_valid, y - (p.col_base + col), st);
          } else if constexpr (kEpi == EPI_LOGP || kEpi == EPI_LOGP_TOP) {
            const float top = logp_chunk(v, col, p.n_valid, y - (p.col_base + col), p.exp_scale, lst);
            if (kEpi == EPI_LOGP_TOP && __any_sync(0xffffffffu, top > ranking.bound)) {
              const int left = p.n_valid - col;   // columns of the chunk that exist
              const int first = col - n_begin * Cfg::kTileN;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (k % 4 == 0 && __any_sync(0xffffffffu, ranking.count > kBeat - 4)) {
                  const RankCut cut = rank_cut(rank_values, rank_columns, ranking.count, p.top_k);
                  if (row_ok) {
                    ranking.count = cut.count;
                    ranking.bound = fmaxf(ranking.bound, cut.bound);
                    if (cut.bound > -INFINITY) atomicMax(bound_at, ordered_bits(cut.bound));
                  }
                }
                if (v[k] > ranking.bound && k < left) {
                  st_shared_f32(rank_values + ranking.count * (BM * 4), v[k]);
                  st_shared_u16(rank_columns + ranking.count * (BM * 2),
                                static_cast<uint32_t>(first + k));
                  ++ranking.count;
                }
              }
            }
          } else {
            const uint32_t box = stg + (nbox & 1u) * Cfg::kStgBytes;
            // the store issued two boxes ago from this buffer has read it
            if (lane == 0) bulk_wait_group_read<1>();
            __syncwarp();
            if constexpr (kEpi == EPI_GRAD) {
              float g[32];
              grad_chunk(v, col, p.n_valid, y - (p.col_base + col), zmax, a, sc, q, g);
              stage_bf16_row(box, lane, g);
            } else if constexpr (kEpi == EPI_LOGP_GRAD) {
              float g[32];
              logp_grad_chunk(v, col, p.n_valid, y - (p.col_base + col), p.inv_t, k4, target, g);
              stage_bf16_row(box, lane, g);
            } else if (p.out_mode == OUT_STORE_BF16) {
              stage_bf16_row(box, lane, v);
            } else {
              stage_f32_row(box, lane, v);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              // rows and columns outside the map are dropped by the store
              const int oy = p.out_row0 + m_blk * Cfg::kTileM + static_cast<int>(rank) * BM +
                             quarter * 32;
              if constexpr (epi_writes_g(kEpi)) tma_store_3d(&G.c, box, col & 63, oy, col >> 6);
              else if (p.out_mode == OUT_ADD_F32) tma_reduce_add_2d(&G.c, box, col, oy);
              else tma_store_2d(&G.c, box, col, oy);
              bulk_commit_group();
            }
            ++nbox;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kCta == 2) mbar_arrive_cluster(acc == 0 ? tempty_leader0 : tempty_leader1);
          else mbar_arrive(tempty_bar(acc));
        }
        if (++acc == Cfg::kAccs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if constexpr (kEpi == EPI_LSE) {
        if (ok) {
          // partial slot of (vocabulary range, 128-row block), independent of the raster
          const int blk128 = m_blk * kCta + static_cast<int>(rank);
          p.part[(static_cast<int64_t>(col_unit) * p.part_stride + blk128) * BM + row] =
              make_float2(st.m, st.s);
          if (row_ok && st.found) p.zt[p.row_base + prow] = st.zt;
        }
      }
      if constexpr (kEpi == EPI_LOGP || kEpi == EPI_LOGP_TOP) {
        if (ok) {
          const int blk128 = m_blk * kCta + static_cast<int>(rank);
          const int64_t slot = (static_cast<int64_t>(col_unit) * p.part_stride + blk128) * BM + row;
          p.part4[slot] = make_float4(lst.p.m, lst.p.s, lst.p.t, 0.f);
          if (row_ok && lst.found) p.zt[p.row_base + prow] = lst.zt;
          if constexpr (kEpi == EPI_LOGP_TOP) {   // in no order: the join sorts them
            const RankCut cut = rank_cut(rank_values, rank_columns, ranking.count, p.top_k);
            if (row_ok && cut.bound > -INFINITY) atomicMax(bound_at, ordered_bits(cut.bound));
            const int n = cut.count;
            const int id0 = p.col_base + n_begin * Cfg::kTileN;
            for (int j = 0; j < p.top_k; ++j)
              p.lists[slot * p.top_k + j] =
                  j < n ? rank_key(ld_shared_f32(rank_values + j * (BM * 4)),
                                   id0 + static_cast<int>(ld_shared_u16(rank_columns + j * (BM * 2))))
                        : 0;
          }
        }
      }
    }
    if (!ok) {
      if (lane == 0) record_status(p0.status, kStatusTimeout);
      *abort_flag = 1;
      // this warp's rows of what is not done become NaN, for callers that do not read the status
      if constexpr (kEpi == EPI_LOGP || kEpi == EPI_LOGP_TOP) {
        for (int u = stop_u; u < total_units; u += num_pairs) {
          int m_blk, n_begin, n_end;
          const int col_unit = unit_tiles<kEpi>(p0, u, m_blk, n_begin, n_end);
          const int64_t slot =
              (static_cast<int64_t>(col_unit) * p0.part_stride + m_blk * kCta + static_cast<int>(rank)) * BM + row;
          p0.part4[slot] = make_float4(__uint_as_float(0x7FC00000u), 0.f, 0.f, 0.f);
          if constexpr (kEpi == EPI_LOGP_TOP)
            for (int j = 0; j < p0.top_k; ++j) p0.lists[slot * p0.top_k + j] = 0;
        }
      } else if constexpr (kEpi == EPI_LOGP_GRAD || kEpi == EPI_F32) {
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        for (uint32_t at = lane * 16u; at < Cfg::kStgBytes; at += 512u)   // NaN in fp32 and in bf16
          st_shared_v4(stg + at, 0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu);
        fence_proxy_async_smem();
        __syncwarp();
        for (int u = stop_u; lane == 0 && u < total_units; u += num_pairs) {
          const bool second = kProducts == 2 && u >= units0;
          const GemmArgs& G = second ? g1 : g0;
          int m_blk, n_begin, n_end;
          unit_tiles<kEpi>(G.p, second ? u - units0 : u, m_blk, n_begin, n_end);
          const int oy = G.p.out_row0 + m_blk * Cfg::kTileM + static_cast<int>(rank) * BM + quarter * 32;
          for (int n_blk = u == stop_u ? stop_n : n_begin; n_blk < n_end; ++n_blk)
            for (int c = 0; c < Cfg::kTileN / 32; ++c) {
              const int col = n_blk * Cfg::kTileN + c * 32;
              if constexpr (epi_writes_g(kEpi)) tma_store_3d(&G.c, stg, col & 63, oy, col >> 6);
              else if (G.p.out_mode == OUT_ADD_F32) tma_reduce_add_2d(&G.c, stg, col, oy);
              else tma_store_2d(&G.c, stg, col, oy);
              bulk_commit_group();
            }
        }
        __syncwarp();
      }
    }
    // every store of this warp has landed before the CTA can exit
    if constexpr (!epi_sums_rows(kEpi)) {
      if (lane == 0) bulk_wait_group_all();
      __syncwarp();
    }
  }

  tc_fence_before();
  if constexpr (kCta == 2) cluster_sync();  // the pair's copies and MMAs have drained
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_cg<kCta>(tmem_base, kTmemCols);
}

// Host-side launch of one instantiation: grid/kCta clusters of kCta CTAs, the tile
// configuration's dynamic shared memory, the products' maps and parameters passed
// by value (g1 is ignored unless kProducts == 2).
template <int kEpi, int kCta, int kFp8, int kWide, int kProducts = 1>
cudaError_t launch_gemm(const GemmArgs& g0, const GemmArgs& g1, int grid, cudaStream_t stream) {
  auto kern = flce_gemm_kernel<kEpi, kCta, kFp8, kWide, kProducts>;
  constexpr size_t smem = TileCfg<kCta, kWide>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, g0, g1);
}

}  // namespace flce
