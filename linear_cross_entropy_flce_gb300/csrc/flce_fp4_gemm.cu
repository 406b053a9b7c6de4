// y = H W^T for matrices in 4-bit floating point, on the block-scaled tensor cores.
//
//   y_nv = h_n w_v sum over blocks b of s_nb t_vb (sum over the block's values of a_i c_i)
//
// with a, c E2M1, s, t the blocks' scales and h, w the rows' (nvfp4). The scales of the blocks go to
// the tensor cores with the operands, from TMEM; the rows' are multiplied in at the end.
//
// The rows of W take the M side of a tile (128 per tcgen05.mma) and the tokens the N side, padded to
// kN = 16 to 384, so that a tile's work follows the tokens there are (above 64, the last tile's to 32s). A ring
// stage holds 256 values of each row, 128 bytes as TMA swizzles them, and the scale bytes of both, which lie in
// memory as tcgen05.cp takes them to TMEM. Up to 256 tokens each CTA streams its own share of W's rows, in whole
// 32s; more tokens go tile by tile, all of a row tile's tokens before the next. From 65 tokens on a cluster pair
// shares a tile of 256 rows, each CTA staging half of the tokens (8192 x 4096 x 128256 nvfp4 by single CTAs
// 1.88 ms, by pairs 1.83, with rows of y 16 bytes at a time 1.60, in boxes 1.51). Tiles of 384 tokens are two MMAs
// on one copy of W's rows; which calls take them is decided in flce_fp4_gemm.h. The scales are copied to TMEM with
// each stage, in the order in which the tensor core takes the MMAs after them.
//
// y in bf16: a warp reads its 32 rows of the accumulator as matrix fragments, so that two tokens' values of a
// row are neighbours in a register, turns 8 x 8 of them at a time on their way to shared memory, and 32 rows of
// 16 tokens leave in a box while the next 16 are made. Rows of y that are not aligned, and fp32, go by columns.
// The next tile's MMAs wait for the accumulator to be read: as it is, up to 256 tokens; 384 are more than the
// registers hold, so they are scaled and narrowed first.
//
// Up to 128 tokens bound by the reads of W: D = 4096, V = 128256 nvfp4 51 us for 1 token, 55 for 64, 56 for 128
// (5.7 to 5.9 TB/s); 74 for 256. Long prompts: 8192 tokens 1.33 to 1.37 ms in short runs and 1.47 to 1.53 under the
// power cap (5.6 to 6.4 PFLOP/s), mxfp4 1.21 and 1.29 (6.7 to 7.1); a library's nvfp4 product, without row scales, 1.20
// and 1.31. Steps are of K = 64, 10.3 PFLOP/s at full clock (this chip also has dense ones of K = 96, at the nominal
// 13.5, which are not used); a stage of 256 tokens takes 262 ns without its loads, of which the steps are 247, and
// 350 with them. Short rows are bound by the outputs: 4000 x 512 x 120000 to fp32 364 us (5.4 TB/s; with the rows'
// scales read only once the tile is done 435), 8000 x 512 x 120000 to bf16 547 us, mxfp4 448 (the library's nvfp4
// 361; in tiles of 256 604 and 507, row by row through shared memory 830 and 601).
#include <cstdint>

#include "flce_blocks.h"
#include "flce_fp4_gemm.h"
#include "flce_gemm_params.h"
#include "flce_launch.cuh"
#include "flce_norm.cuh"
#include "ptx.cuh"

namespace flce {

namespace {

constexpr int kEpilogue = 8;              // warps of the epilogue, then the copying one and the MMAs'
constexpr int kCopyWarp = kEpilogue, kMmaWarp = kEpilogue + 1;
constexpr int kThreads = (kEpilogue + 2) * 32;
constexpr int kOutTokens = kFp4OutTokens;

template <int kN, int kNv, int kCta>
struct Cfg {
  static constexpr int kRows = 128 * kCta;                  // of W in a tile
  static constexpr int kTokenTiles = (kN + 127) / 128;
  // of a CTA: its 128 rows of W, its share of the tokens, the scales of its rows and of all tokens
  static constexpr uint32_t kABytes = 128 * 128;
  static constexpr uint32_t kBBytes = kN / kCta * 128;
  static constexpr uint32_t kSf = kNv ? 2048 : 1024;        // scale bytes of 128 rows' 256 values
  static constexpr int kBlocks = kSf / 512;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSf * (1 + kTokenTiles);
  // of an epilogue warp: twice kOutTokens rows on their way out, its tokens' row scales
  static constexpr uint32_t kOutBytes = kN >= 64 ? 2 * kOutTokens * 64 + (kNv ? kN / 2 * 4 : 0) : 0;
  static constexpr int kFit = static_cast<int>((225 * 1024 - kEpilogue * kOutBytes) / kStageBytes);
  static constexpr int kStages = kFit > 10 ? 10 : kFit;
  static constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + kEpilogue * kOutBytes + 512;
  static constexpr int kAcc = kN >= 256 ? 1 : 2;            // accumulators
  // TMEM: the accumulators, then kSfBuffers times the scales of a stage
  static constexpr int kSfCols = kBlocks * 4 * (1 + kTokenTiles);
  static constexpr int kSfBuffers = 2;
  static constexpr int kCols = kAcc * kN + kSfBuffers * kSfCols;
  static constexpr uint32_t kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM has 512 columns");
  static_assert(kSmemBytes <= 232448, "more dynamic shared memory than a CTA may have");
  static_assert(kStageBytes % 1024 == 0, "swizzled boxes begin at multiples of 1024 bytes");
};

// 512 bytes of scales (32 rows of 16) to 4 TMEM columns, the same in each quarter of the lanes; in a
// pair, each CTA's to its own.
template <int kCta>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem) {
  // no swizzle; groups of 8 rows are 128 bytes apart
  const uint64_t desc = static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
                        (1ull << 46);
  if constexpr (kCta == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <int kNv, int kCta>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
#define FLCE_MMA_FP4(form)                                                                                \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\ttcgen05.mma." form                           \
               " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                           \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                              \
               : "memory")
  if constexpr (kNv && kCta == 2) FLCE_MMA_FP4("cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (kNv) FLCE_MMA_FP4("cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (kCta == 2) FLCE_MMA_FP4("cta_group::2.kind::mxf4.block_scale.scale_vec::2X");
  else FLCE_MMA_FP4("cta_group::1.kind::mxf4.block_scale.scale_vec::2X");
#undef FLCE_MMA_FP4
}

// Instruction descriptor of a 128 kCta x n x 64 step: E2M1 operands, both K-major; scales E4M3 (nvfp4) or
// powers of two; sf: which of the four bytes of a row's scale word the step begins with.
template <int kNv, int kCta>
__device__ __forceinline__ constexpr uint32_t fp4_idesc(int n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((kNv ? 0u : 1u) << 23) |
         ((128u * kCta >> 4) << 24) | (sf << 29);
}

// 16 lanes x 32 columns: of columns 8 k and on, lane l holds columns 2 (l % 4) and the next, of rows l / 4
// (r[4 k], r[4 k + 1]) and l / 4 + 8 (the two after them)
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// four 8 x 8 matrices of 16 bits, held as above, to shared memory by columns: lane l gives the place of
// column l % 8 of matrix l / 8
__device__ __forceinline__ void st_matrices_by_column(uint32_t a, uint32_t m0, uint32_t m1, uint32_t m2,
                                                      uint32_t m3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(m0),
               "r"(m1), "r"(m2), "r"(m3)
               : "memory");
}

template <int kCols>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  if constexpr (kCols >= 32) {
#pragma unroll
    for (int c = 0; c < kCols; c += 32) {
      uint32_t(&v)[32] = *reinterpret_cast<uint32_t(*)[32]>(r + c);
      tmem_ld_32x32b_x32(taddr + c, v);
    }
  } else if constexpr (kCols == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    static_assert(kCols == 8, "8, 16 or whole 32s");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  }
}

// The tiles of a CTA (or a pair): rows [row, row_end) of W within the kRows from row / kRows * kRows on,
// tokens from `token` on, one after another.
template <int kN, int kRows>
struct Tiles {
  int row, row_end, token;
  int last_row;        // share: where its rows end
  int64_t unit, units; // tiles: the next one
  int step, token_tiles, V, N;
  bool share;
  __device__ Tiles(const Fp4GemmParams& p, int index, int count) {
    V = p.V;
    N = p.N;
    share = p.N <= kN;
    token = 0;
    token_tiles = (p.N + kN - 1) / kN;
    step = count;
    if (share) {
      const int64_t groups = (p.V + 31) / 32;
      row = static_cast<int>(groups * index / count * 32);
      last_row = min(p.V, static_cast<int>(groups * (index + 1) / count * 32));
      row_end = min(last_row, row / kRows * kRows + kRows);
    } else {
      units = static_cast<int64_t>((p.V + kRows - 1) / kRows) * token_tiles;
      unit = index;
      place();
    }
  }
  __device__ void place() {
    row = static_cast<int>(unit / token_tiles) * kRows;
    row_end = min(V, row + kRows);
    token = static_cast<int>(unit % token_tiles) * kN;
  }
  __device__ bool more() const { return share ? row < last_row : unit < units; }
  __device__ void next() {
    if (share) {
      row = row_end;
      row_end = min(last_row, row + kRows);
    } else {
      unit += step;
      if (unit < units) place();
    }
  }
  // the tokens of an MMA, of the tile's from `first` on: the last tile's are as few as its tokens, in 32s, 16 from
  // either CTA of a pair
  __device__ int width(int first, int most) const {
    return kRows == 128 ? most : max(0, min(most, (N - token - first + 31) / 32 * 32));
  }
  // the 32s of rows, counted from CTA `rank`'s 128, that its copies take: [first, end)
  __device__ void quarters(int rank, int& first, int& end) const {
    const int base = row / kRows * kRows + rank * 128;
    first = max(0, (row - base) / 32);
    end = min(4, (row_end - base + 31) / 32);
    if (end < first) end = first;
  }
};

// kCta = 2: cluster pairs; each CTA stages its 128 rows of W and half of the tokens, and the even one
// issues the MMAs of both.
template <int kN, int kNv, int kBf16, int kCta>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ Fp4Maps maps, const Fp4GemmParams p) {
  using C = Cfg<kN, kNv, kCta>;
  using At = Tiles<kN, C::kRows>;
  constexpr bool kCl = kCta == 2;   // waits acquire at cluster scope
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * C::kStageBytes + kEpilogue * C::kOutBytes);
  // full[kStages] | empty[kStages] | tfull[2] | tempty[2] | drain
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kCl ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int index = static_cast<int>(blockIdx.x) / kCta, count = static_cast<int>(gridDim.x) / kCta;
  const uint32_t stage0 = smem_u32(smem);
  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + kStages + s); };
  auto tfull_bar = [&](int a) { return smem_u32(bars + 2 * kStages + a); };
  auto tempty_bar = [&](int a) { return smem_u32(bars + 2 * kStages + 2 + a); };
  const uint32_t drain_bar = smem_u32(bars + 2 * kStages + 4);
  // of a stage: W's codes | the tokens' | W's scales | the tokens' scales
  constexpr uint32_t kOffB = C::kABytes, kOffSfA = C::kStageBytes - C::kSf * (1 + C::kTokenTiles),
                     kOffSfB = kOffSfA + C::kSf;
  if (threadIdx.x == 0) {
    // the even CTA's full[s] counts the copies of both
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kEpilogue * kCta);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.h);
    tma_prefetch_desc(&maps.w_scales);
    tma_prefetch_desc(&maps.h_scales);
  }
  // the barriers of both CTAs are there before either touches the other's
  if constexpr (kCl) cluster_sync();
  else __syncthreads();
  if (warp == kMmaWarp) {
    tmem_alloc_cg<kCta>(smem_u32(tmem_holder), C::kTmemCols);
    tmem_relinquish_cg<kCta>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  wait_for_launch_before();   // nothing of the operands is read, nothing of y written before
  const uint64_t tmo = p.timeout_ns;
  const volatile int no_abort = 0;
  auto fail = [&]() {
    if (lane == 0 && p.status != nullptr) atomicCAS(reinterpret_cast<int*>(p.status), 0, kStatusTimeout);
    *abort_flag = 1;
  };

  if (warp == kCopyWarp) {
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    bool ok = true;
    const uint64_t pol_w = make_l2_policy(p.N <= kN ? 1 : 0), pol_h = make_l2_policy(2);
    for (At at(p, index, count); ok && at.more(); at.next()) {
      const int base = at.row / C::kRows * C::kRows + static_cast<int>(rank) * 128;
      int q0, q1;
      at.quarters(static_cast<int>(rank), q0, q1);
      uint32_t bytes = 0;   // of a stage, both CTAs'
#pragma unroll
      for (int c = 0; c < kCta; ++c) {
        int f, e;
        at.quarters(c, f, e);
        bytes += static_cast<uint32_t>(e - f) * 32u * 128u + C::kBBytes + C::kSf * (1 + C::kTokenTiles);
      }
      for (int ks = 0; ks < p.stages; ++ks) {
        const bool free_ok = mbar_wait_bounded<kCl>(empty_bar(stage), phase ^ 1u, tmo, abort_flag);
        if (!__all_sync(0xffffffffu, free_ok)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t at_stage = stage0 + stage * C::kStageBytes;
          if (leader) mbar_arrive_expect_tx(full_bar(stage), bytes);
          // copies complete on the even CTA's barrier
          const uint32_t fb = kCl ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
          auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t pol) {
            if constexpr (kCl) tma_load_2d_pair(dst, map, x, y, fb, pol);
            else tma_load_2d_hint(dst, map, x, y, fb, pol);
          };
          if (q0 == 0 && q1 == 4) {
            load(at_stage, &maps.w, ks * 128, base, pol_w);
          } else {
            for (int q = q0; q < q1; ++q) load(at_stage + q * 32 * 128, &maps.w32, ks * 128, base + q * 32, pol_w);
          }
          if constexpr (kN > 256) {   // both MMAs' halves
            const int one = at.token + static_cast<int>(rank) * (at.width(0, 256) / 2);
            load(at_stage + kOffB, &maps.h, ks * 128, one, pol_h);
            load(at_stage + kOffB + 64 * 128, &maps.h, ks * 128, one + 64, pol_h);
            load(at_stage + kOffB + 128 * 128, &maps.h, ks * 128,
                 at.token + 256 + static_cast<int>(rank) * (at.width(256, 128) / 2), pol_h);
          } else {
            load(at_stage + kOffB, &maps.h, ks * 128, at.token + static_cast<int>(rank) * (at.width(0, kN) / kCta),
                 pol_h);
          }
          load(at_stage + kOffSfA, &maps.w_scales, 0, (base / 128 * p.stages + ks) * C::kBlocks, pol_w);
#pragma unroll
          for (int tt = 0; tt < C::kTokenTiles; ++tt)
            load(at_stage + kOffSfB + tt * C::kSf, &maps.h_scales, 0,
                 ((at.token / 128 + tt) * p.stages + ks) * C::kBlocks, pol_h);
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
    if (!ok) fail();
    // The copies that were issued land before the CTAs' memory is given back. The even CTA's barriers
    // count the odd one's too; after an abort the odd CTA may have issued copies that the even one never
    // armed, so it waits far longer than a copy takes.
    if (leader) {
      for (int s = 0; s < kStages; ++s)
        if (issued_mask & (1u << s))
          mbar_wait_bounded<kCl>(full_bar(s), (issued_par >> s) & 1u, 1000000000ull, &no_abort);
    } else if (!ok || *abort_flag) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) {
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp && leader) {
    int stage = 0, acc = 0, buffer = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued_any = false;
    for (At at(p, index, count); ok && at.more(); at.next()) {
      const bool acc_ok = mbar_wait_bounded<kCl>(tempty_bar(acc), acc_phase ^ 1u, tmo, abort_flag);
      if (!__all_sync(0xffffffffu, acc_ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kN);
      constexpr int kFirst = kN > 256 ? 256 : kN;
      const int width = at.width(0, kFirst);
      [[maybe_unused]] const int beyond = at.width(kFirst, kN - kFirst);
      for (int ks = 0; ks < p.stages; ++ks) {
        const bool full_ok = mbar_wait_bounded<kCl>(full_bar(stage), phase, tmo, abort_flag);
        if (!__all_sync(0xffffffffu, full_ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t at_stage = stage0 + stage * C::kStageBytes;
          const uint32_t sfa = tmem_base + C::kAcc * kN + buffer * C::kSfCols;
          const uint32_t sfb = sfa + C::kBlocks * 4;
#pragma unroll
          for (int b = 0; b < C::kBlocks; ++b) {
            copy_scales<kCta>(sfa + b * 4, at_stage + kOffSfA + b * 512);
#pragma unroll
            for (int tt = 0; tt < C::kTokenTiles; ++tt)
              copy_scales<kCta>(sfb + (b * C::kTokenTiles + tt) * 4, at_stage + kOffSfB + tt * C::kSf + b * 512);
          }
#pragma unroll
          for (int k = 0; k < kFp4Stage / 64; ++k) {
            const int b = kNv ? k : k / 2;
            const uint32_t sf = kNv ? 0u : static_cast<uint32_t>(k % 2 * 2);
            mma_fp4<kNv, kCta>(d_tmem, make_sw128_desc(at_stage + k * 32, 16, 1024),
                               make_sw128_desc(at_stage + kOffB + k * 32, 16, 1024), fp4_idesc<kNv, kCta>(width, sf),
                               sfa + b * 4, sfb + b * C::kTokenTiles * 4, (ks | k) != 0 ? 1u : 0u);
            if constexpr (kN > 256) {
              if (beyond > 0)
                mma_fp4<kNv, kCta>(d_tmem + 256, make_sw128_desc(at_stage + k * 32, 16, 1024),
                                   make_sw128_desc(at_stage + kOffB + 128 * 128 + k * 32, 16, 1024),
                                   fp4_idesc<kNv, kCta>(beyond, sf), sfa + b * 4,
                                   sfb + (b * C::kTokenTiles + 2) * 4, (ks | k) != 0 ? 1u : 0u);
            }
          }
          umma_commit_pair<kCta>(empty_bar(stage));   // frees the stage in both CTAs
        }
        __syncwarp();
        issued_any = true;
        buffer ^= 1;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) umma_commit_pair<kCta>(tfull_bar(acc));
      __syncwarp();
      if (++acc == C::kAcc) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok) fail();
    if (issued_any) {   // every MMA is done before TMEM is freed
      if (elect_one()) umma_commit_cg<kCta>(drain_bar);
      __syncwarp();
      mbar_wait_bounded(drain_bar, 0, 1000000000ull, &no_abort);
    }
    __syncwarp();
  } else if (warp < kEpilogue) {
    constexpr int kHalf = kN / 2;   // columns of a warp
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t from = (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * kHalf);
    const uint32_t s_out = stage0 + kStages * C::kStageBytes + warp * (2 * kOutTokens * 64);
    [[maybe_unused]] float* const s_rows = reinterpret_cast<float*>(
        smem + kStages * C::kStageBytes + kEpilogue * (2 * kOutTokens * 64) + warp * (kHalf * 4));
    int acc = 0;
    uint32_t acc_phase = 0;
    // this lane's row of a tile, and whether the tile has it
    auto row_of = [&](const At& at, bool& mine) {
      const int r = at.row / C::kRows * C::kRows + static_cast<int>(rank) * 128 + quarter * 32 + lane;
      mine = r >= at.row && r < at.row_end;
      return r;
    };
    for (At at(p, index, count); at.more(); at.next()) {
      bool mine;
      const int r = row_of(at, mine);
      const int first = at.token + half * kHalf;
      const int tokens = min(kHalf, p.N - first);
      // where all of a warp's 32 rows of bf16 are there, they meet in shared memory and leave in boxes
      const bool wide = fp4_boxes(kN, kBf16) && p.wide && __all_sync(0xffffffffu, mine);
      // the rows' scales, on their way while the tile is: of this lane's row, or of the four that it holds then
      [[maybe_unused]] float w_row[4], h_row[(kHalf + 31) / 32];
      if constexpr (kNv) {
        if (wide) {
#pragma unroll
          for (int m = 0; m < 4; ++m) w_row[m] = p.w_rows[r - lane + (lane >> 2) + 8 * m];
        } else {
          w_row[0] = mine ? p.w_rows[r] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < (kHalf + 31) / 32; ++k)
          h_row[k] = k * 32 + lane < tokens ? p.h_rows[first + k * 32 + lane] : 0.f;
      }
      int got = 0;
      if (lane == 0) got = mbar_wait_bounded<kCl>(tfull_bar(acc), acc_phase, tmo, abort_flag) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        fail();
        // this warp's part of what is not done becomes NaN, for callers that do not read the status
        for (; at.more(); at.next()) {
          const int row = row_of(at, mine);
          if (!mine) continue;
          for (int n = at.token + half * kHalf; n < min(p.N, at.token + half * kHalf + kHalf); ++n) {
            if (kBf16) static_cast<uint16_t*>(p.y)[n * p.ldy + row] = 0x7FC0u;
            else static_cast<float*>(p.y)[n * p.ldy + row] = __uint_as_float(0x7FC00000u);
          }
        }
        break;
      }
      tc_fence_after();
      const uint32_t at_tmem = tmem_base + from + static_cast<uint32_t>(acc * kN);
      auto read = [&]() {   // the accumulator has been read
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kCl) mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));
          else mbar_arrive(tempty_bar(acc));
        }
        if (++acc == C::kAcc) {
          acc = 0;
          acc_phase ^= 1u;
        }
      };
      if (tokens <= 0) {   // the other half's warps have them all
        read();
        continue;
      }
      if constexpr (kNv && kHalf >= 32) {
        __syncwarp();   // the tile before has read them
#pragma unroll
        for (int k = 0; k < kHalf / 32; ++k) s_rows[k * 32 + lane] = h_row[k];
      }
      if constexpr (fp4_boxes(kN, kBf16)) {
        if (wide) {
          // 32 rows of 8 tokens, two tokens of a row in a register, rows l / 4 + 8 m of lane l
          constexpr int kHeld = kHalf <= 128 ? kHalf : 32;   // tokens held as they are
          uint32_t v[2][kHeld / 2];   // rows 0 to 15 of the warp's 32, and the rest
          [[maybe_unused]] uint32_t done[kHalf / 8][4];
          auto load = [&](int first_column) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
              for (int c = 0; c < kHeld; c += 32)
                tmem_ld_16x256b_x4(at_tmem + (static_cast<uint32_t>(u * 16) << 16) + first_column + c,
                                   *reinterpret_cast<uint32_t(*)[16]>(&v[u][c / 2]));
            }
          };
          // tokens c to c + 7 of those from `held` on that are in v
          auto narrow = [&](int held, int c, uint32_t (&out)[4]) {
            float2 h = make_float2(1.f, 1.f);
            if constexpr (kNv) h = *reinterpret_cast<const float2*>(s_rows + held + c + (lane & 3) * 2);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const int k = c / 2 + (m & 1) * 2;
              float a = __uint_as_float(v[m >> 1][k]), b = __uint_as_float(v[m >> 1][k + 1]);
              if constexpr (kNv) {
                split(mul2(mul2(pair(a, b), pair(w_row[m], w_row[m])), pair(h.x, h.y)), a, b);
              }
              out[m] = pack_bf16x2(a, b);
            }
          };
          if constexpr (kHeld == kHalf) {
            load(0);
          } else {   // more than the registers take: narrowed as they are read
            __syncwarp();
#pragma unroll
            for (int held = 0; held < kHalf; held += kHeld) {
              load(held);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < kHeld; c += 8) narrow(held, c, done[(held + c) / 8]);
            }
          }
          read();
          // a token's 64 bytes, its four 16-byte pieces as the copy swizzles them: eight tokens are on all banks
          const uint32_t put = static_cast<uint32_t>((lane & 7) * 64 + ((lane >> 3) ^ ((lane >> 1) & 3)) * 16);
#pragma unroll
          for (int c0 = 0; c0 < kHalf; c0 += kOutTokens) {
            if (c0 >= tokens) break;
            const uint32_t place = s_out + c0 / kOutTokens % 2 * (kOutTokens * 64);
            // one place after the other: the copy from this one, two steps ago, has read it. A tile begins at the first
            // place, from which the one before took its last box where it had an odd number of them, so all have to be
            // read (as they long are; a place that goes on from tile to tile took 580 us instead of 547 for 8000 x 512 x
            // 120000 nvfp4, in whose registers it had no room)
            if (lane == 0) {
              if (c0 == 0) bulk_wait_group_read<0>();
              else bulk_wait_group_read<1>();
            }
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kOutTokens; c += 8) {
              uint32_t out[4];
              if constexpr (kHeld == kHalf) {
                narrow(0, c0 + c, out);
              } else {
#pragma unroll
                for (int m = 0; m < 4; ++m) out[m] = done[(c0 + c) / 8][m];
              }
              st_matrices_by_column(place + c * 64 + put, out[0], out[1], out[2], out[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {   // tokens behind the last are not written
              tma_store_2d(&maps.y, place, r, first + c0);
              bulk_commit_group();
            }
          }
          continue;
        }
      }
      if constexpr (kHalf > 128) {   // the warp in which W's rows end: 32 tokens at a time
        __syncwarp();
        for (int c0 = 0; c0 < tokens; c0 += 32) {
          uint32_t v[32];
          tmem_ld<32>(at_tmem + c0, v);
          tmem_wait_ld();
          uint16_t* y = static_cast<uint16_t*>(p.y) + (first + c0) * p.ldy + r;
#pragma unroll
          for (int c = 0; c < 32; ++c, y += p.ldy) {
            float o = __uint_as_float(v[c]);
            if constexpr (kNv) o = o * w_row[0] * s_rows[c0 + c];
            if (mine && c0 + c < tokens) *y = static_cast<uint16_t>(pack_bf16x2(o, 0.f) & 0xFFFFu);
          }
        }
        read();
        continue;
      }
      uint32_t v[kHalf];
      tmem_ld<kHalf>(at_tmem, v);
      read();
      if constexpr (kHalf >= 32) {
        // some tokens at a time
#pragma unroll
        for (int c0 = 0; c0 < kHalf; c0 += kOutTokens) {
          if (c0 >= tokens) break;
          float o[kOutTokens];
#pragma unroll
          for (int c = 0; c < kOutTokens; c += 4) {
            float4 h = make_float4(1.f, 1.f, 1.f, 1.f);
            if constexpr (kNv) h = *reinterpret_cast<const float4*>(s_rows + c0 + c);
            const float hs[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[c + e] = __uint_as_float(v[c0 + c + e]);
              if constexpr (kNv) o[c + e] = o[c + e] * w_row[0] * hs[e];
            }
          }
          const int n = min(kOutTokens, tokens - c0);
          if (!mine) continue;
          if constexpr (kBf16) {
            uint16_t* y = static_cast<uint16_t*>(p.y) + (first + c0) * p.ldy + r;
#pragma unroll
            for (int c = 0; c < kOutTokens; ++c, y += p.ldy)
              if (c < n) *y = static_cast<uint16_t>(pack_bf16x2(o[c], 0.f) & 0xFFFFu);
          } else {
            float* y = static_cast<float*>(p.y) + (first + c0) * p.ldy + r;
#pragma unroll
            for (int c = 0; c < kOutTokens; ++c, y += p.ldy)
              if (c < n) *y = o[c];
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < kHalf; ++c) {
          float o = __uint_as_float(v[c]);
          if constexpr (kNv) o = o * w_row[0] * __shfl_sync(0xffffffffu, h_row[0], c);
          if (c < tokens && mine) {
            const int64_t to = (first + c) * p.ldy + r;
            if constexpr (kBf16) static_cast<uint16_t*>(p.y)[to] = static_cast<uint16_t>(pack_bf16x2(o, 0.f) & 0xFFFFu);
            else static_cast<float*>(p.y)[to] = o;
          }
        }
      }
    }
    if constexpr (fp4_boxes(kN, kBf16)) {
      if (lane == 0) bulk_wait_group_all();
    }
  }
  tc_fence_before();
  if constexpr (kCl) cluster_sync();   // the pair's copies and MMAs are done
  else __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_cg<kCta>(tmem_base, C::kTmemCols);
}

template <int kN, int kNv, int kBf16, int kCta>
cudaError_t launch(const Fp4Maps& maps, const Fp4GemmParams& p, int sms, cudaStream_t stream) {
  using C = Cfg<kN, kNv, kCta>;
  auto kern = fp4_gemm_kernel<kN, kNv, kBf16, kCta>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmemBytes));
  if (e != cudaSuccess) return e;
  const int64_t units = p.N <= kN ? (p.V + 31) / 32
                                  : static_cast<int64_t>((p.V + C::kRows - 1) / C::kRows) * ((p.N + kN - 1) / kN);
  const int most = sms / kCta;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((units < most ? units : most) * kCta));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // the tokens' quantisation, most often the launch before, lets this one set itself up meanwhile
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

// (384 tokens only for y in bf16 and boxes)
template <int kN, int kCta>
cudaError_t launch_types(int nv, int bf16, const Fp4Maps& maps, const Fp4GemmParams& p, int sms,
                         cudaStream_t stream) {
  if constexpr (kN > 256) {
    if (!bf16 || !p.wide) return cudaErrorInvalidValue;
    return nv ? launch<kN, 1, 1, kCta>(maps, p, sms, stream) : launch<kN, 0, 1, kCta>(maps, p, sms, stream);
  } else if (nv) {
    return bf16 ? launch<kN, 1, 1, kCta>(maps, p, sms, stream) : launch<kN, 1, 0, kCta>(maps, p, sms, stream);
  } else {
    return bf16 ? launch<kN, 0, 1, kCta>(maps, p, sms, stream) : launch<kN, 0, 0, kCta>(maps, p, sms, stream);
  }
}

}  // namespace

cudaError_t launch_fp4_gemm(int kn, int nv, int bf16, const Fp4Maps& maps, const Fp4GemmParams& p, int sms,
                            cudaStream_t stream) {
  switch (kn) {
    case 16: return launch_types<16, fp4_ctas(16)>(nv, bf16, maps, p, sms, stream);
    case 32: return launch_types<32, fp4_ctas(32)>(nv, bf16, maps, p, sms, stream);
    case 64: return launch_types<64, fp4_ctas(64)>(nv, bf16, maps, p, sms, stream);
    case 128: return launch_types<128, fp4_ctas(128)>(nv, bf16, maps, p, sms, stream);
    case 256: return launch_types<256, fp4_ctas(256)>(nv, bf16, maps, p, sms, stream);
    case 384: return launch_types<384, fp4_ctas(384)>(nv, bf16, maps, p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace flce
