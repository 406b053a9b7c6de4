// Arithmetic of the block-scaled formats.
//
// Scales that are powers of two come from the bits of the block's largest magnitude: with amax =
// 1.m 2^E and the format's largest value 1.75 2^8 (E4M3) or 1.5 2^2 (E2M1), the smallest e with
// amax <= largest 2^e is E - 8 (or E - 2), and one more where 1.m is above 1.75 (or 1.5). Dividing
// by 2^e is then exact, and the hardware's conversion rounds once, to nearest even. Magnitudes
// are compared as the integers their bits are, by which infinities and NaN come out largest.
#pragma once

#include <cstdint>

#include "flce_blocks.h"
#include "flce_norm.cuh"

namespace flce {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;

// The byte e + 127 of a block with largest magnitude amax (its bits): kExp and kMant from the
// format's largest value, whose mantissa has nothing beyond kMant: what is above it carries into the exponent.
// 255 for an infinity or NaN, 0 where amax is that small.
template <int kExp, uint32_t kMant>
__device__ __forceinline__ uint32_t power_scale_byte(uint32_t amax) {
  const int b = static_cast<int>((amax + (0x7FFFFFu - kMant)) >> 23) - kExp;
  return amax >= kInfBits ? 255u : static_cast<uint32_t>(max(b, 0));
}
__device__ __forceinline__ uint32_t e4m3_scale_byte(uint32_t amax) {
  return power_scale_byte<8, 0x600000u>(amax);
}

// 2^(byte - 127), NaN for 255; and its reciprocal (of a byte up to 253).
__device__ __forceinline__ float power_of_byte(uint32_t b) {
  uint32_t two;   // bf16, exact
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(b)));
  return __uint_as_float(two << 16);
}
__device__ __forceinline__ float inverse_power_of_byte(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Two values to E4M3, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 codes (the low 16 bits) to fp32.
__device__ __forceinline__ void widen_e4m3x2(uint32_t codes, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

// Four codes of values times inv.
__device__ __forceinline__ uint32_t e4m3x4(const float* v, float inv) {
  const uint64_t by = pair(inv, inv);
  float q[4];
  split(mul2(pair(v[0], v[1]), by), q[0], q[1]);
  split(mul2(pair(v[2], v[3]), by), q[2], q[3]);
  return e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16;
}

// Eight values to E2M1, the first in the lowest bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight E2M1 codes to fp32.
__device__ __forceinline__ void widen_e2m1x8(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(v[2 * k]), "=f"(v[2 * k + 1])
        : "r"(h[k]));
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The bits of the largest magnitude of VW values.
template <int VW>
__device__ __forceinline__ uint32_t largest_bits(const float (&v)[VW]) {
  uint32_t m = magnitude(v[0]);
#pragma unroll
  for (int e = 1; e < VW; ++e) m = max(m, magnitude(v[e]));
  return m;
}

// The same of bf16 as loaded, two at a time (a NaN comes out as one).
template <int kWords>
__device__ __forceinline__ uint32_t largest_bits_bf16(const uint32_t* w) {
  uint32_t m;
  asm("abs.bf16x2 %0, %1;" : "=r"(m) : "r"(w[0]));
#pragma unroll
  for (int k = 1; k < kWords; ++k)
    asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %1;\n\tmax.NaN.bf16x2 %0, %0, a;\n\t}" : "+r"(m) : "r"(w[k]));
  return max(m & 0xFFFF0000u, m << 16);
}

// Over groups of kLanes neighbouring lanes (a power of two).
template <int kLanes>
__device__ __forceinline__ uint32_t largest_of_lanes(uint32_t m) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Rows that do not allow wide accesses: a warp's 32 VW neighbouring elements go through shared memory,
// so that its accesses of 2 or 4 bytes lie side by side while each lane has VW neighbours.
// (A lane's are VW + 1 words apart, an odd number.)
template <int VW>
constexpr int kWarpStage = 32 * (VW + 1);   // floats of a warp

// in: elements first + lane, first + 32 + lane, ... of the row, 0 from D on.
template <int kBf16, int VW>
__device__ __forceinline__ void load_apart(const void* row, int first, int D, float (&in)[VW]) {
#pragma unroll
  for (int k = 0; k < VW; ++k) {
    const int i = first + k * 32 + static_cast<int>(threadIdx.x & 31);
    in[k] = i < D ? load_as_f32(row, i, kBf16) : 0.f;
  }
}
// v: the elements [lane VW, + VW) of those.
template <int VW>
__device__ __forceinline__ void to_neighbours(const float (&in)[VW], float* stage, float (&v)[VW]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int k = 0; k < VW; ++k) stage[k * 32 + lane + (k * 32 + lane) / VW] = in[k];
  __syncwarp();
#pragma unroll
  for (int e = 0; e < VW; ++e) v[e] = stage[lane * (VW + 1) + e];
}

// Both, the other way round.
template <int kBf16, int VW>
__device__ __forceinline__ void store_staged(void* row, int first, int D, float* stage, const float (&v)[VW]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int e = 0; e < VW; ++e) stage[lane * (VW + 1) + e] = v[e];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < VW; ++k) {
    const int i = k * 32 + lane;
    if (first + i < D) store_from_f32(row, first + i, stage[i + i / VW], kBf16);
  }
}

// 16 values as loaded.
template <int kBf16>
struct Chunk {
  uint4 w[kBf16 ? 2 : 4];
  __device__ void load_if(const uint8_t* row, int i, bool ok) {
#pragma unroll
    for (int k = 0; k < (kBf16 ? 2 : 4); ++k)
      w[k] = ok ? reinterpret_cast<const uint4*>(row + i * 16 * (kBf16 ? 2 : 4))[k] : make_uint4(0, 0, 0, 0);
  }
  __device__ void narrow(const float (&v)[16]) {   // of values that are kBf16's
#pragma unroll
    for (int k = 0; k < (kBf16 ? 2 : 4); ++k) {
      constexpr int n = kBf16 ? 8 : 4;
      float q[n];
#pragma unroll
      for (int e = 0; e < n; ++e) q[e] = v[k * n + e];
      w[k] = Pack<kBf16, n>::narrow(q);
    }
  }
  __device__ void widen(float (&v)[16]) const {
#pragma unroll
    for (int k = 0; k < (kBf16 ? 2 : 4); ++k) {
      constexpr int n = kBf16 ? 8 : 4;
      float q[n];
      Pack<kBf16, n>::widen(w[k], q);
#pragma unroll
      for (int e = 0; e < n; ++e) v[k * n + e] = q[e];
    }
  }
  __device__ uint32_t largest() const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (kBf16) {
      return largest_bits_bf16<8>(u);
    } else {
      uint32_t m = u[0] & 0x7FFFFFFFu;
#pragma unroll
      for (int e = 1; e < 16; ++e) m = max(m, u[e] & 0x7FFFFFFFu);
      return m;
    }
  }
};

// Chunks t, t + R, ... of a row of D values, 0 behind it; all lanes of the warp. kWhole: 16-byte accesses.
template <int kBf16, int kWhole, int n>
__device__ __forceinline__ void load_chunks(const uint8_t* row, int t, int R, int D, float* stage,
                                            Chunk<kBf16> (&c)[n]) {
  if constexpr (kWhole) {
#pragma unroll
    for (int k = 0; k < n; ++k) c[k].load_if(row, t + k * R, (t + k * R) * 16 + 16 <= D);
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const int i = (t + k * R) * 16;
      if (i < D && i + 16 > D) {   // the chunk in which the row ends
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = i + e < D ? load_as_f32(row, i + e, kBf16) : 0.f;
        c[k].narrow(v);
      }
    }
  } else {
    float in[n][16];   // all loads first
#pragma unroll
    for (int k = 0; k < n; ++k)
      load_apart<kBf16, 16>(row, (t + k * R - static_cast<int>(threadIdx.x & 31)) * 16, D, in[k]);
#pragma unroll
    for (int k = 0; k < n; ++k) {
      float v[16];
      to_neighbours(in[k], stage, v);
      c[k].narrow(v);
    }
  }
}

inline bool whole_vectors(const void* x, int bf16, int64_t ldx) {
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * (bf16 ? 2 : 4) % 16 == 0;
}

}  // namespace
}  // namespace flce
