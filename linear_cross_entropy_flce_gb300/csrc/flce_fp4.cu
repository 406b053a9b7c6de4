// 4-bit floating point: quantisation and the values back.
//
// mxfp4: 32 values share 2^e, e the smallest >= -127 with amax <= 6 2^e.
// nvfp4: 16 values share an E4M3 scale s = rn(amax / 6 / g), g the row's smallest power of two >=
// 2^-126 with the row's largest magnitude <= 6 448 g; values x / (s g).
// Codes are E2M1, rounded once, to nearest even (nvfp4's largest may saturate where s was rounded
// down).
//
// A group of R threads holds a row in registers, eight neighbouring values a vector, so that it is
// read once for the row's and the blocks' largest magnitudes and the codes; rows of more than 32768
// values are read again instead. 1 / s is rounded, so the quotient x r is corrected by its
// residual, which makes it x / s rounded once (Markstein's theorem): a value halfway between two codes
// stays there. (In fp32 no other quotient is rounded onto such a place: its distance from it is at
// least the quotient's own last place.)
#include <cstdint>

#include "flce_blocks.cuh"
#include "flce_norm.cuh"

namespace flce {

namespace {

constexpr int kFp4Threads = 256;
constexpr int kFp4Vectors = 4;   // of a row in a thread's registers at most

// Vector i (8 values from 8 i on) of a row of D; zeros behind it.
template <int kBf16, int kWhole>
__device__ __forceinline__ void load_vector(const uint8_t* row, int i, int D, float (&v)[8]) {
  if (kWhole && i * 8 + 8 <= D) {
    Param<kBf16, 8> raw;
    raw.load(row, i * 8, 0.f);
    raw.widen(v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = i * 8 + e < D ? load_as_f32(row, i * 8 + e, kBf16) : 0.f;
  }
}

// The largest finite magnitude.
__device__ __forceinline__ uint32_t largest_finite(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = magnitude(v[e]);
    m = max(m, b < kInfBits ? b : 0u);
  }
  return m;
}

// One vector's codes and its block's scale byte. All lanes of the warp.
template <int kNv>
__device__ __forceinline__ uint32_t quantize_vector(float (&v)[8], float inv_row, uint32_t& byte) {
  const uint32_t amax = largest_of_lanes<kNv ? 2 : 4>(largest_bits(v));
  const bool finite = amax < kInfBits;
  if constexpr (kNv) {
    byte = finite ? e4m3x2(__fdiv_rn(__uint_as_float(amax), 6.f) * inv_row, 0.f) & 0xFFu : 0x7Fu;
    float s, none;
    widen_e4m3x2(finite ? byte : 0u, s, none);
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = finite ? v[e] * inv_row : 0.f;
      const float q = x * r;
      v[e] = copysignf(fmaf(fmaf(-q, s, x), r, q), x);   // the correction makes +0 of -0
    }
  } else {
    byte = power_scale_byte<2, 0x400000u>(amax);
    const float inv = finite ? inverse_power_of_byte(byte) : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = finite ? v[e] * inv : 0.f;
  }
  return e2m1x8(v);
}

// The bytes of four neighbouring blocks, in the first of their lanes.
template <int kNv>
__device__ __forceinline__ uint32_t four_bytes(uint32_t byte) {
  constexpr int kLanes = kNv ? 2 : 4;   // of a block
  uint32_t w = byte << (8 * ((threadIdx.x / kLanes) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, kLanes);
  w |= __shfl_xor_sync(0xffffffffu, w, 2 * kLanes);
  return w;
}

// Rows up to the next multiple of 128: those past N have scales alone, 0. kHeld: vectors of a row in
// a thread's registers; 0: read twice.
template <int kBf16, int kNv, int kWhole, int kHeld>
__global__ void __launch_bounds__(1024)
    quantize_fp4_kernel(const void* x, int64_t ldx, int N, int D, uint8_t* codes, uint8_t* scales,
                        float* row_scales, int R) {
  __shared__ uint32_t s_max[32];
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kLanes4 = (kNv ? 2 : 4) * 4;   // threads of four blocks
  const int t = static_cast<int>(threadIdx.x) % R;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / R) + threadIdx.x / R;
  const bool live = row < N;
  const uint8_t* const from = static_cast<const uint8_t*>(x) + row * ldx * kElt;
  const int width = live ? D : 0;
  const int nvec = static_cast<int>(fp4_stages(D)) * (kFp4Stage / 8);
  const int code_bytes = static_cast<int>(fp4_code_bytes(D));
  float held[kHeld > 0 ? kHeld : 1][8];
  if constexpr (kHeld > 0) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) load_vector<kBf16, kWhole>(from, t + k * R, width, held[k]);
  }
  float inv_row = 1.f;
  if constexpr (kNv) {
    uint32_t m = 0;
    if constexpr (kHeld > 0) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) m = largest_finite(held[k], m);
    } else {
      for (int i = t; i < nvec; i += R) {
        float v[8];
        load_vector<kBf16, kWhole>(from, i, width, v);
        m = largest_finite(v, m);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (R > 32) {
      const int warp = static_cast<int>(threadIdx.x) >> 5, per = R >> 5;
      if ((threadIdx.x & 31) == 0) s_max[warp] = m;
      __syncthreads();
      for (int w = 0; w < per; ++w) m = max(m, s_max[warp / per * per + w]);
    }
    uint32_t byte = power_scale_byte<11, 0x280000u>(m);
    byte = m == 0 ? 127u : byte < 1u ? 1u : byte;
    inv_row = inverse_power_of_byte(byte);
    if (t == 0 && live) row_scales[row] = power_of_byte(byte);
  }
  auto put = [&](int i, float (&v)[8]) {
    uint32_t byte;
    const uint32_t c = quantize_vector<kNv>(v, inv_row, byte);
    // (a block behind the row, whose largest is 0, has the byte 0 too)
    const uint32_t w = four_bytes<kNv>(byte);
    if (i >= nvec) return;
    if (live && i * 4 < code_bytes) *reinterpret_cast<uint32_t*>(codes + row * code_bytes + i * 4) = c;
    if (t % kLanes4 == 0) *reinterpret_cast<uint32_t*>(scales + fp4_scale_at(row, i / kLanes4, D, kNv)) = w;
  };
  if constexpr (kHeld > 0) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) put(t + k * R, held[k]);
  } else {
    for (int i = t; i < (nvec + R - 1) / R * R; i += R) {   // whole warps, for the shuffles
      float v[8];
      load_vector<kBf16, kWhole>(from, i, width, v);
      put(i, v);
    }
  }
}

template <int kBf16, int kNv>
__global__ void __launch_bounds__(kFp4Threads)
    dequantize_fp4_kernel(const uint8_t* codes, const uint8_t* scales, const float* row_scales, int N, int D,
                          void* x, int64_t ldx, int X, int whole) {
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kBlock = fp4_block(kNv);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kFp4Threads / X) + threadIdx.x / X;
  if (row >= N) return;
  const int t = static_cast<int>(threadIdx.x) % X;
  uint8_t* const to = static_cast<uint8_t*>(x) + row * ldx * kElt;
  const float row_scale = kNv ? row_scales[row] : 1.f;
  const int first = static_cast<int>(blockIdx.y) * X * kFp4Vectors + t;
  uint32_t c[kFp4Vectors], byte[kFp4Vectors];
#pragma unroll
  for (int k = 0; k < kFp4Vectors; ++k) {
    const int i = first + k * X;
    if (i * 8 < D) {
      const int block = i * 8 / kBlock;
      c[k] = *reinterpret_cast<const uint32_t*>(codes + row * fp4_code_bytes(D) + i * 4);
      byte[k] = scales[fp4_scale_at(row, block / 4, D, kNv) + block % 4];
    }
  }
#pragma unroll
  for (int k = 0; k < kFp4Vectors; ++k) {
    const int i = first + k * X;
    if (i * 8 >= D) break;
    float s, none;
    if (kNv) widen_e4m3x2(byte[k], s, none);
    else s = power_of_byte(byte[k]);
    float v[8];
    widen_e2m1x8(c[k], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * s * row_scale;
    if (whole && i * 8 + 8 <= D) {
      Param<kBf16, 8> out;
      out.narrow(v);
      out.save(to, i * 8);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i * 8 + e < D) store_from_f32(to, i * 8 + e, v[e], kBf16);
    }
  }
}

bool whole_vectors(const void* x, int bf16, int64_t ldx) {
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * (bf16 ? 2 : 4) % 16 == 0;
}

// f with a, b, c as compile-time constants.
template <typename F>
cudaError_t with_flags(bool a, bool b, bool c, F&& f) {
  using One = std::integral_constant<int, 1>;
  using Zero = std::integral_constant<int, 0>;
  auto third = [&](auto x, auto y) { return c ? f(x, y, One{}) : f(x, y, Zero{}); };
  auto second = [&](auto x) { return b ? third(x, One{}) : third(x, Zero{}); };
  return a ? second(One{}) : second(Zero{});
}

}  // namespace

cudaError_t launch_quantize_fp4(const void* x, int bf16, int64_t ldx, int N, int D, int nv, uint8_t* codes,
                                uint8_t* scales, float* row_scales, int sms, cudaStream_t stream) {
  const int nvec = static_cast<int>(fp4_stages(D)) * (kFp4Stage / 8);
  const int64_t rows = (static_cast<int64_t>(N) + kFp4RowTile - 1) / kFp4RowTile * kFp4RowTile;
  // Threads of a row: enough for kFp4Vectors vectors each, and more while the rows alone do not
  // fill the GPU.
  int R = 32;
  while (R < 1024 && R * kFp4Vectors < nvec) R *= 2;
  while (R < 1024 && R < nvec && N * static_cast<int64_t>(R) < static_cast<int64_t>(sms) * 512) R *= 2;
  const int block = R < kFp4Threads ? kFp4Threads : R;
  const unsigned grid = static_cast<unsigned>((rows * R + block - 1) / block);
  return with_flags(bf16 != 0, nv != 0, whole_vectors(x, bf16, ldx), [&](auto b, auto n, auto w) {
    auto go = [&](auto kern) {
      kern<<<grid, block, 0, stream>>>(x, ldx, N, D, codes, scales, row_scales, R);
      return cudaGetLastError();
    };
    const int per = (nvec + R - 1) / R;
    if (per <= 1) return go(quantize_fp4_kernel<b(), n(), w(), 1>);
    if (per <= 2) return go(quantize_fp4_kernel<b(), n(), w(), 2>);
    if (per <= kFp4Vectors) return go(quantize_fp4_kernel<b(), n(), w(), kFp4Vectors>);
    return go(quantize_fp4_kernel<b(), n(), w(), 0>);
  });
}

cudaError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* row_scales, int N,
                                  int D, int nv, void* x, int bf16, int64_t ldx, cudaStream_t stream) {
  const int nvec = (D + 7) / 8;
  int X = 4;
  while (X < kFp4Threads && X < nvec) X *= 2;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(N) * X + kFp4Threads - 1) / kFp4Threads),
                  static_cast<unsigned>((nvec + X * kFp4Vectors - 1) / (X * kFp4Vectors)));
  return with_flags(bf16 != 0, nv != 0, false, [&](auto b, auto n, auto) {
    dequantize_fp4_kernel<b(), n()><<<grid, kFp4Threads, 0, stream>>>(codes, scales, row_scales, N, D, x, ldx, X,
                                                                      whole_vectors(x, bf16, ldx));
    return cudaGetLastError();
  });
}

}  // namespace flce
