// y = H W^T for matrices in 4-bit floating point, on the block-scaled tensor cores.
//
//   y_nv = h_n w_v sum over blocks b of s_nb t_vb (sum over the block's values of a_i c_i)
//
// with a, c E2M1, s, t the blocks' scales and h, w the rows' (nvfp4). The scales of the blocks go to
// the tensor cores with the operands, from TMEM; the rows' are multiplied in at the end.
//
// The rows of W take the M side of a tile (128 per tcgen05.mma) and the tokens the N side, padded to
// kN = 16 to 256, so that a tile's work follows the tokens there are. A ring stage holds 256 values of
// each row, 128 bytes as TMA swizzles them, and the scale bytes of both, which lie in memory as
// tcgen05.cp takes them to TMEM. Up to 256 tokens each CTA streams its own share of W's rows, in whole
// 32s; more tokens go tile by tile, all of a row tile's tokens before the next.
#include <cstdint>

#include "flce_blocks.h"
#include "flce_fp4_gemm.h"
#include "flce_gemm_params.h"
#include "ptx.cuh"

namespace flce {

namespace {

constexpr int kWarps = 12;   // TMA, MMA, two without work, eight of the epilogue
constexpr int kThreads = kWarps * 32;
constexpr int kEpilogue = 8;

template <int kN, int kNv>
struct Cfg {
  static constexpr int kTokenTiles = (kN + 127) / 128;
  static constexpr uint32_t kABytes = 128 * 128;
  static constexpr uint32_t kBBytes = kN * 128;
  static constexpr uint32_t kSf = kNv ? 2048 : 1024;        // scale bytes of 128 rows' 256 values
  static constexpr int kBlocks = kSf / 512;
  static constexpr uint32_t kStageBytes = kABytes + (kBBytes < 1024 ? 1024 : kBBytes) + kSf * (1 + kTokenTiles);
  static constexpr int kFit = static_cast<int>((224 * 1024) / kStageBytes);
  static constexpr int kStages = kFit > 10 ? 10 : kFit;
  static constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + 512;
  static constexpr int kAcc = kN == 256 ? 1 : 2;            // accumulators
  // TMEM: the accumulators, then kSfBuffers times the scales of a stage
  static constexpr int kSfCols = kBlocks * 4 * (1 + kTokenTiles);
  static constexpr int kSfBuffers = 2;
  static constexpr int kCols = kAcc * kN + kSfBuffers * kSfCols;
  static constexpr uint32_t kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM has 512 columns");
  static_assert(kSmemBytes <= 232448, "more dynamic shared memory than a CTA may have");
  static_assert(kStageBytes % 1024 == 0, "swizzled boxes begin at multiples of 1024 bytes");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// 512 bytes of scales (32 rows of 16) to 4 TMEM columns, the same in each quarter of the lanes.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem) {
  // no swizzle; groups of 8 rows are 128 bytes apart
  const uint64_t desc = static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
                        (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <int kNv>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of a 128 x kN x 64 step: E2M1 operands, both K-major; scales E4M3 (nvfp4) or
// powers of two; sf: which of the four bytes of a row's scale word the step begins with.
template <int kN, int kNv>
__device__ __forceinline__ constexpr uint32_t fp4_idesc(uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kN >> 3) << 17) | ((kNv ? 0u : 1u) << 23) |
         ((128u >> 4) << 24) | (sf << 29);
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

// The tiles of a CTA: (rows [row, row_end) of W within the 128 from row / 128 * 128 on, tokens from
// `token` on), one after another.
template <int kN>
struct Tiles {
  int row, row_end, token;
  int last_row;        // share: where this CTA's rows end
  int64_t unit, units; // tiles: the next one
  int token_tiles, V;
  bool share;
  __device__ Tiles(const Fp4GemmParams& p) {
    V = p.V;
    share = p.N <= kN;
    token = 0;
    token_tiles = (p.N + kN - 1) / kN;
    if (share) {
      const int64_t groups = (p.V + 31) / 32;
      row = static_cast<int>(groups * blockIdx.x / gridDim.x * 32);
      last_row = min(p.V, static_cast<int>(groups * (blockIdx.x + 1) / gridDim.x * 32));
      row_end = min(last_row, row / 128 * 128 + 128);
    } else {
      units = static_cast<int64_t>((p.V + 127) / 128) * token_tiles;
      unit = blockIdx.x;
      place();
    }
  }
  __device__ void place() {
    row = static_cast<int>(unit / token_tiles) * 128;
    row_end = min(V, row + 128);
    token = static_cast<int>(unit % token_tiles) * kN;
  }
  __device__ bool more() const { return share ? row < last_row : unit < units; }
  __device__ void next() {
    if (share) {
      row = row_end;
      row_end = min(last_row, row + 128);
    } else {
      unit += gridDim.x;
      if (unit < units) place();
    }
  }
};

template <int kN, int kNv, int kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mW32,
                    const __grid_constant__ CUtensorMap mH, const Fp4GemmParams p) {
  using C = Cfg<kN, kNv>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * C::kStageBytes);
  // full[kStages] | empty[kStages] | tfull[2] | tempty[2] | drain
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kEpilogue);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mW);
    tma_prefetch_desc(&mW32);
    tma_prefetch_desc(&mH);
  }
  __syncthreads();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  const uint64_t tmo = p.timeout_ns;
  const volatile int no_abort = 0;
  auto fail = [&]() {
    if (lane == 0 && p.status != nullptr) atomicCAS(reinterpret_cast<int*>(p.status), 0, kStatusTimeout);
    *abort_flag = 1;
  };

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    bool ok = true;
    const uint64_t pol_w = make_l2_policy(p.N <= kN ? 1 : 0), pol_h = make_l2_policy(2);
    for (Tiles<kN> at(p); ok && at.more(); at.next()) {
      const int tile = at.row / 128;
      const int q0 = at.row % 128 / 32, q1 = (at.row_end - tile * 128 + 31) / 32;   // its 32s of rows
      const bool whole = q0 == 0 && q1 == 4;
      const uint32_t w_bytes = static_cast<uint32_t>(q1 - q0) * 32u * 128u;
      // the tokens' scale tiles that there are (one at least)
      const int sf_tiles = C::kTokenTiles == 1 || at.token + 128 >= p.N ? 1 : 2;
      const uint8_t* const sf_w = p.w_scales + static_cast<int64_t>(tile) * p.stages * C::kSf;
      const uint8_t* const sf_h = p.h_scales + static_cast<int64_t>(at.token / 128) * p.stages * C::kSf;
      for (int ks = 0; ks < p.stages; ++ks) {
        const bool free_ok = mbar_wait_bounded(empty_bar(stage), phase ^ 1u, tmo, abort_flag);
        if (!__all_sync(0xffffffffu, free_ok)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t fb = full_bar(stage), at_stage = stage0 + stage * C::kStageBytes;
          mbar_arrive_expect_tx(fb, w_bytes + C::kBBytes + C::kSf * (1 + sf_tiles));
          if (whole) {
            tma_load_2d_hint(at_stage, &mW, ks * 128, tile * 128, fb, pol_w);
          } else {
            for (int q = q0; q < q1; ++q)
              tma_load_2d_hint(at_stage + q * 32 * 128, &mW32, ks * 128, tile * 128 + q * 32, fb, pol_w);
          }
          tma_load_2d_hint(at_stage + kOffB, &mH, ks * 128, at.token, fb, pol_h);
          bulk_load(at_stage + kOffSfA, sf_w + ks * C::kSf, C::kSf, fb);
          for (int tt = 0; tt < sf_tiles; ++tt)
            bulk_load(at_stage + kOffSfB + tt * C::kSf,
                      sf_h + (static_cast<int64_t>(tt) * p.stages + ks) * C::kSf, C::kSf, fb);
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
    // the copies that were issued land before the CTA's memory is given back
    for (int s = 0; s < kStages; ++s)
      if (issued_mask & (1u << s)) mbar_wait_bounded(full_bar(s), (issued_par >> s) & 1u, 1000000000ull, &no_abort);
    __syncwarp();
  } else if (warp == 1) {
    int stage = 0, acc = 0, buffer = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued_any = false;
    for (Tiles<kN> at(p); ok && at.more(); at.next()) {
      const bool acc_ok = mbar_wait_bounded(tempty_bar(acc), acc_phase ^ 1u, tmo, abort_flag);
      if (!__all_sync(0xffffffffu, acc_ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kN);
      for (int ks = 0; ks < p.stages; ++ks) {
        const bool full_ok = mbar_wait_bounded(full_bar(stage), phase, tmo, abort_flag);
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
            copy_scales(sfa + b * 4, at_stage + kOffSfA + b * 512);
#pragma unroll
            for (int tt = 0; tt < C::kTokenTiles; ++tt)
              copy_scales(sfb + (b * C::kTokenTiles + tt) * 4, at_stage + kOffSfB + tt * C::kSf + b * 512);
          }
#pragma unroll
          for (int k = 0; k < kFp4Stage / 64; ++k) {
            const int b = kNv ? k : k / 2;
            const uint32_t sf = kNv ? 0u : static_cast<uint32_t>(k % 2 * 2);
            mma_fp4<kNv>(d_tmem, make_sw128_desc(at_stage + k * 32, 16, 1024),
                         make_sw128_desc(at_stage + kOffB + k * 32, 16, 1024), fp4_idesc<kN, kNv>(sf), sfa + b * 4,
                         sfb + b * C::kTokenTiles * 4, (ks | k) != 0 ? 1u : 0u);
          }
          umma_commit_cg<1>(empty_bar(stage));
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
      if (elect_one()) umma_commit_cg<1>(tfull_bar(acc));
      __syncwarp();
      if (++acc == C::kAcc) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok) fail();
    if (issued_any) {   // every MMA is done before TMEM is freed
      if (elect_one()) umma_commit_cg<1>(drain_bar);
      __syncwarp();
      mbar_wait_bounded(drain_bar, 0, 1000000000ull, &no_abort);
    }
    __syncwarp();
  } else if (warp >= kWarps - kEpilogue) {
    constexpr int kHalf = kN / 2;   // columns of a warp
    const int quarter = warp & 3, half = (warp - (kWarps - kEpilogue)) >> 2;
    const uint32_t from = (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * kHalf);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (Tiles<kN> at(p); at.more(); at.next()) {
      const int r = at.row / 128 * 128 + quarter * 32 + lane;
      const bool mine = r >= at.row && r < at.row_end;
      const int first = at.token + half * kHalf;
      const int tokens = min(kHalf, p.N - first);
      int got = 0;
      if (lane == 0) got = mbar_wait_bounded(tfull_bar(acc), acc_phase, tmo, abort_flag) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        fail();
        // this warp's part of what is not done becomes NaN, for callers that do not read the status
        for (; at.more(); at.next()) {
          const int row = at.row / 128 * 128 + quarter * 32 + lane;
          if (row < at.row || row >= at.row_end) continue;
          for (int n = at.token + half * kHalf; n < min(p.N, at.token + half * kHalf + kHalf); ++n) {
            if (kBf16) static_cast<uint16_t*>(p.y)[n * p.ldy + row] = 0x7FC0u;
            else static_cast<float*>(p.y)[n * p.ldy + row] = __uint_as_float(0x7FC00000u);
          }
        }
        break;
      }
      tc_fence_after();
      uint32_t v[kHalf];
      tmem_ld<kHalf>(tmem_base + from + static_cast<uint32_t>(acc * kN), v);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
      if (++acc == C::kAcc) {
        acc = 0;
        acc_phase ^= 1u;
      }
      [[maybe_unused]] float w_row = 1.f, h_row[(kHalf + 31) / 32];
      if constexpr (kNv) {
        if (mine) w_row = p.w_rows[r];
#pragma unroll
        for (int k = 0; k < (kHalf + 31) / 32; ++k)
          h_row[k] = k * 32 + lane < tokens ? p.h_rows[first + k * 32 + lane] : 0.f;
      }
#pragma unroll
      for (int c = 0; c < kHalf; ++c) {
        float o = __uint_as_float(v[c]);
        if constexpr (kNv) o = o * w_row * __shfl_sync(0xffffffffu, h_row[c / 32], c % 32);
        if (c < tokens && mine) {
          const int64_t to = (first + c) * p.ldy + r;
          if constexpr (kBf16) static_cast<uint16_t*>(p.y)[to] = static_cast<uint16_t>(pack_bf16x2(o, 0.f) & 0xFFFFu);
          else static_cast<float*>(p.y)[to] = o;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, C::kTmemCols);
}

template <int kN, int kNv, int kBf16>
cudaError_t launch(const CUtensorMap& mW, const CUtensorMap& mW32, const CUtensorMap& mH, const Fp4GemmParams& p,
                   int sms, cudaStream_t stream) {
  constexpr size_t smem = Cfg<kN, kNv>::kSmemBytes;
  auto kern = fp4_gemm_kernel<kN, kNv, kBf16>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t units = p.N <= kN ? (p.V + 31) / 32
                                  : static_cast<int64_t>((p.V + 127) / 128) * ((p.N + kN - 1) / kN);
  kern<<<static_cast<unsigned>(units < sms ? units : sms), kThreads, smem, stream>>>(mW, mW32, mH, p);
  return cudaGetLastError();
}

template <int kN>
cudaError_t launch_types(int nv, int bf16, const CUtensorMap& mW, const CUtensorMap& mW32, const CUtensorMap& mH,
                         const Fp4GemmParams& p, int sms, cudaStream_t stream) {
  if (nv) return bf16 ? launch<kN, 1, 1>(mW, mW32, mH, p, sms, stream) : launch<kN, 1, 0>(mW, mW32, mH, p, sms, stream);
  return bf16 ? launch<kN, 0, 1>(mW, mW32, mH, p, sms, stream) : launch<kN, 0, 0>(mW, mW32, mH, p, sms, stream);
}

}  // namespace

cudaError_t launch_fp4_gemm(int kn, int nv, int bf16, const CUtensorMap& mW, const CUtensorMap& mW32,
                            const CUtensorMap& mH, const Fp4GemmParams& p, int sms, cudaStream_t stream) {
  switch (kn) {
    case 16: return launch_types<16>(nv, bf16, mW, mW32, mH, p, sms, stream);
    case 32: return launch_types<32>(nv, bf16, mW, mW32, mH, p, sms, stream);
    case 64: return launch_types<64>(nv, bf16, mW, mW32, mH, p, sms, stream);
    case 128: return launch_types<128>(nv, bf16, mW, mW32, mH, p, sms, stream);
    default: return launch_types<256>(nv, bf16, mW, mW32, mH, p, sms, stream);
  }
}

}  // namespace flce
