// The product of two 4-bit matrices (flce_fp4_gemm.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace flce {

struct Fp4GemmParams {
  int N, V;                 // rows of H (tokens), rows of W
  int stages;               // of 256 values
  const float *h_rows, *w_rows;   // row scales, or null
  void* y;                  // [N][ldy], fp32 or bf16
  int64_t ldy;
  int wide;                 // y takes boxes by maps.y
  int64_t timeout_ns;
  int32_t* status;
};

// Tokens of a tile for N of them, and the CTAs that share it.
inline int fp4_tile(int64_t N) { return N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : N <= 128 ? 128 : 256; }
// 384 tokens instead of 256, where y goes in boxes: a sixth less to read per product, but longer turns. Taken where
// all turns' tokens are at most 4 % more (mxfp4, whose ring is as deep in either, 12 %). In us with 256 / 384: 8192 x 4096 x
// 128256 nvfp4 1518 / 1482, mxfp4 1388 / 1288; 3000 x 4096 x 100000 442 / 422; 2048 x 4096 x 128256 (13 % more) 364 /
// 390; 512 x 4096 x 100000 88 / 102; and for fewer tokens 300 x 4096 x 100000 78 / 78, x 30000 32 / 38.
inline int fp4_wide_tile(int64_t N, int64_t V, int sms, int nv) {
  auto turns = [&](int kn) {
    const int64_t tiles = (V + 255) / 256 * ((N + kn - 1) / kn), pairs = sms / 2;
    return (tiles + pairs - 1) / pairs * kn;
  };
  return N > 384 && turns(384) * 25 <= turns(256) * (nv ? 26 : 28) ? 384 : fp4_tile(N);
}
constexpr int fp4_ctas(int kn) { return kn >= 128 ? 2 : 1; }

// W's codes in boxes of 128 bytes x 128 and x 32 rows, H's in boxes of 128 bytes x kn / ctas rows, both
// (64 where kn is 384) with 128-byte swizzle; the scales' groups of 512 bytes in boxes of those of 256 values; y in bf16, where
// fp4_boxes and the alignment say so, in boxes of 32 x kFp4OutTokens with 64-byte swizzle.
constexpr int kFp4OutTokens = 16;
constexpr bool fp4_boxes(int kn, int bf16) { return bf16 && kn >= 64; }
struct Fp4Maps {
  CUtensorMap w, w32, h, w_scales, h_scales, y;
};

// y = H W^T in tiles of kn tokens: fp4_tile(p.N), or 384 where fp4_wide_tile says so, which takes y in bf16,
// p.wide and H's boxes of 64 rows. Any other kn is cudaErrorInvalidValue.
cudaError_t launch_fp4_gemm(int kn, int nv, int bf16, const Fp4Maps& maps, const Fp4GemmParams& p, int sms,
                            cudaStream_t stream);

}  // namespace flce
