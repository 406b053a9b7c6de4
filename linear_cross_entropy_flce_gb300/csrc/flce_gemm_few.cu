// Logits of a few tokens, Z = H W^T in fp32, for the log probabilities of a decoding batch.
//
// With N tokens the product has to read W once (V D 2 bytes) and little else, so the kernel
// is built around that stream. The rows of W take the M side of the tensor cores' tile
// (128 vocabulary ids per tcgen05.mma) and the tokens the N side, padded to kN = 16, 32, 64
// or 128: the work of a tile follows the tokens there are, where the large GEMM's tile of
// 256 tokens would spend as long on one token as reading W takes. Every CTA streams its
// own contiguous share of W's rows (in multiples of 16, so that the shares differ by at
// most 16 rows) through a ring of TMA boxes; the accumulators of two tiles alternate in TMEM.
//
// Each tile also needs the tokens' K block, a few rows that all SMs want at the same time:
// 152 SMs on one row's 128-byte pieces took 960 us for one token where W alone takes 155. So
// the tokens are first copied to a padded array of 128 rows in 128 / kN copies, and each CTA
// reads one of the copies.
//
// Z goes to the workspace (N rows; it stays in L2) for the row kernel to read.
//
// Bound by the reads of W: D = 4096, V = 128256 (1.05 GB, 155 us at the copy rate) takes 166 us
// with the row kernel for 1 token, 173 for 64, 192 for 128.
#include <cstdint>

#include "flce_gemm_few.h"
#include "ptx.cuh"

namespace flce {

namespace {

constexpr int kFewThreads = 192;

template <int kN>
struct FewCfg {
  static constexpr int kSub = 2;   // K blocks per ring stage
  static constexpr uint32_t kABytes = BM * BK * 2;
  static constexpr uint32_t kBBytes = kN * BK * 2;
  static constexpr uint32_t kSubBytes = kABytes + kBBytes;
  static constexpr uint32_t kStageBytes = kSub * kSubBytes;
  static constexpr int kStages = static_cast<int>(205 * 1024 / kStageBytes);
  static constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + 256;
  static constexpr uint32_t kTmemCols = 2 * kN < 32 ? 32 : 2 * kN;
  static_assert(kSmemBytes <= 232448, "more dynamic shared memory than a CTA may have");
};

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// mW: W in boxes of 64 x 128, mW16: the same in boxes of 64 x 16 (a share's last tile);
// mH: the tokens in boxes of 64 x kN.
template <int kN>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_logits_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mW16,
                      const __grid_constant__ CUtensorMap mH, const FewParams p) {
  using Cfg = FewCfg<kN>;
  constexpr int kStages = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * Cfg::kStageBytes);
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
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mW);
    tma_prefetch_desc(&mW16);
    tma_prefetch_desc(&mH);
  }
  __syncthreads();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  const uint64_t tmo = p.timeout_ns;
  // this CTA's rows of W
  const int64_t groups = (p.V + 15) / 16;
  const int row0 = static_cast<int>(groups * blockIdx.x / gridDim.x * 16);
  const int row1 = min(p.V, static_cast<int>(groups * (blockIdx.x + 1) / gridDim.x * 16));
  const int k_stages = (p.k_blocks + Cfg::kSub - 1) / Cfg::kSub;
  const volatile int no_abort = 0;
  auto fail = [&]() {
    if (lane == 0 && p.status != nullptr)
      atomicCAS(reinterpret_cast<int*>(p.status), 0, kStatusTimeout);
    *abort_flag = 1;
  };

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    bool ok = true;
    const uint64_t pol_w = make_l2_policy(1), pol_h = make_l2_policy(2);
    const int h_row = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.copies)) * kN;
    for (int row = row0; ok && row < row1; row += BM) {
      const int boxes16 = min(BM, row1 - row + 15) / 16;
      const bool whole = row1 - row >= BM;
      const uint32_t w_bytes = whole ? Cfg::kABytes : static_cast<uint32_t>(boxes16) * 16u * BK * 2u;
      for (int ks = 0; ks < k_stages; ++ks) {
        const bool free_ok = mbar_wait_bounded(empty_bar(stage), phase ^ 1u, tmo, abort_flag);
        if (!__all_sync(0xffffffffu, free_ok)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const int nsub = min(Cfg::kSub, p.k_blocks - ks * Cfg::kSub);
          const uint32_t fb = full_bar(stage);
          mbar_arrive_expect_tx(fb, static_cast<uint32_t>(nsub) * (w_bytes + Cfg::kBBytes));
#pragma unroll
          for (int sub = 0; sub < Cfg::kSub; ++sub) {
            if (sub >= nsub) break;
            const int kx = (ks * Cfg::kSub + sub) * BK;
            const uint32_t sa = stage0 + stage * Cfg::kStageBytes + sub * Cfg::kSubBytes;
            if (whole) {
              tma_load_2d_hint(sa, &mW, kx, row, fb, pol_w);
            } else {
              for (int b = 0; b < boxes16; ++b)
                tma_load_2d_hint(sa + b * (16 * BK * 2), &mW16, kx, row + 16 * b, fb, pol_w);
            }
            tma_load_2d_hint(sa + Cfg::kABytes, &mH, kx, h_row, fb, pol_h);
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
    if (!ok) fail();
    // the copies that were issued land before the CTA's memory is given back
    for (int s = 0; s < kStages; ++s)
      if (issued_mask & (1u << s))
        mbar_wait_bounded(full_bar(s), (issued_par >> s) & 1u, 1000000000ull, &no_abort);
    __syncwarp();
  } else if (warp == 1) {
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued_any = false;
    constexpr uint32_t idesc = make_idesc_bf16_f32(BM, kN, 0, 0);
    for (int row = row0; ok && row < row1; row += BM) {
      const bool acc_ok = mbar_wait_bounded(tempty_bar(acc), acc_phase ^ 1u, tmo, abort_flag);
      if (!__all_sync(0xffffffffu, acc_ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kN);
      for (int ks = 0; ks < k_stages; ++ks) {
        const bool full_ok = mbar_wait_bounded(full_bar(stage), phase, tmo, abort_flag);
        if (!__all_sync(0xffffffffu, full_ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int nsub = min(Cfg::kSub, p.k_blocks - ks * Cfg::kSub);
        if (elect_one()) {
#pragma unroll
          for (int sub = 0; sub < Cfg::kSub; ++sub) {
            if (sub >= nsub) break;
            const uint32_t sa = stage0 + stage * Cfg::kStageBytes + sub * Cfg::kSubBytes;
#pragma unroll
            for (int k = 0; k < BK / UK; ++k)
              umma_bf16_cg<1>(d_tmem, make_sw128_desc(sa + k * (UK * 2), 16, 1024),
                              make_sw128_desc(sa + Cfg::kABytes + k * (UK * 2), 16, 1024), idesc,
                              (ks | sub | k) != 0 ? 1u : 0u);
          }
          umma_commit_cg<1>(empty_bar(stage));
        }
        __syncwarp();
        issued_any = true;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) umma_commit_cg<1>(tfull_bar(acc));
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (!ok) fail();
    if (issued_any) {   // every MMA is done before TMEM is freed
      if (elect_one()) umma_commit_cg<1>(drain_bar);   // the lane that issued them
      __syncwarp();
      mbar_wait_bounded(drain_bar, 0, 1000000000ull, &no_abort);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int row = row0; row < row1; row += BM) {
      int got = 0;
      if (lane == 0) got = mbar_wait_bounded(tfull_bar(acc), acc_phase, tmo, abort_flag) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        fail();
        // this warp's rows of what is not done become NaN, for callers that do not read the status
        for (int r = row + quarter * 32 + lane; r < row1; r += BM)
          for (int j = 0; j < p.N; ++j) p.z[r + j * p.ldz] = __uint_as_float(0x7FC00000u);
        break;
      }
      tc_fence_after();
      const int r = row + quarter * 32 + lane;
      float* out = p.z + r;
#pragma unroll 1
      for (int c = 0; c < kN && c < p.N; c += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tmem_base + lane_addr + static_cast<uint32_t>(acc * kN + c), v);
        tmem_wait_ld();
        if (r < row1) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < p.N) out[static_cast<int64_t>(c + j) * p.ldz] = __uint_as_float(v[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::kTmemCols);
}

// out row r = token r % per (zeros past N), in rows of D bf16 (D % 8 == 0).
__global__ void pad_tokens_kernel(const uint4* __restrict__ H, int N, int vecs, int per,
                                  uint4* __restrict__ out) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= vecs) return;
  const int token = static_cast<int>(blockIdx.y) % per;
  out[static_cast<int64_t>(blockIdx.y) * vecs + i] =
      token < N ? H[static_cast<int64_t>(token) * vecs + i] : make_uint4(0, 0, 0, 0);
}

template <int kN>
cudaError_t launch_few(const CUtensorMap& mW, const CUtensorMap& mW16, const CUtensorMap& mH,
                       const FewParams& p, int grid, cudaStream_t stream) {
  constexpr size_t smem = FewCfg<kN>::kSmemBytes;
  const cudaError_t e = cudaFuncSetAttribute(
      few_logits_kernel<kN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  few_logits_kernel<kN><<<grid, kFewThreads, smem, stream>>>(mW, mW16, mH, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pad_tokens(const uint16_t* H, int N, int D, int per, uint16_t* out,
                              cudaStream_t stream) {
  const int vecs = D / 8;
  pad_tokens_kernel<<<dim3(static_cast<unsigned>((vecs + 127) / 128), kFewPadRows), 128, 0, stream>>>(
      reinterpret_cast<const uint4*>(H), N, vecs, per, reinterpret_cast<uint4*>(out));
  return cudaGetLastError();
}

cudaError_t launch_few_logits(int kn, const CUtensorMap& mW, const CUtensorMap& mW16,
                              const CUtensorMap& mH, const FewParams& p, int sms,
                              cudaStream_t stream) {
  const int groups = (p.V + 15) / 16;
  const int grid = groups < sms ? groups : sms;
  switch (kn) {
    case 16: return launch_few<16>(mW, mW16, mH, p, grid, stream);
    case 32: return launch_few<32>(mW, mW16, mH, p, grid, stream);
    case 64: return launch_few<64>(mW, mW16, mH, p, grid, stream);
    default: return launch_few<128>(mW, mW16, mH, p, grid, stream);
  }
}

}  // namespace flce
