// 4-bit floating point: quantisation and the values back.
//
// mxfp4: 32 values share 2^e, e the smallest >= -127 with amax <= 6 2^e.
// nvfp4: 16 values share an E4M3 scale s = rn(amax / 6 / g), g the row's smallest power of two >=
// 2^-126 with the row's largest magnitude <= 6 448 g; values x / (s g).
// Codes are E2M1, rounded once, to nearest even (nvfp4's largest may saturate where s was rounded
// down).
//
// A group of R threads holds a row in registers, 16 neighbouring values a chunk, so that it is
// read once for the row's and the blocks' largest magnitudes and the codes; rows of more than 32768
// values (16384 through shared memory) are read again instead. Rows that do not allow 16-byte accesses come through shared memory, a
// warp's 512 values at a time. 1 / s is taken in two parts, r and its
// rest, so that x r + x rest is x / s to within 2^-43, rounded once: a value halfway between two codes
// stays there. (And no other quotient is rounded onto such a place: its distance from it is more than
// half the quotient's own last place.) amax / 6 is rounded in the same way, so that the scale's rounding is the one
// that counts.
//
// Bound by instructions for nvfp4 (so two values an instruction), by bytes for mxfp4 and for the values back: 128256 x
// 4096 bf16 233, 186 and 208 us (the bytes 201, 198); 8192 x 4096 18.8 and 14.7; 64128 x 4096 fp32 194; 3001 x 1111
// fp32 7.7, 5.5 and 4.2 (the bytes 2.3; rows that are not whole 16 bytes are read 2 or 4 bytes at a time); one row of
// 4096 1.9 and 1.6. The quotient corrected by its residual instead (three operations a value) 317.
#include <cstdint>

#include "flce_blocks.cuh"
#include "flce_launch.cuh"

namespace flce {

namespace {

constexpr int kFp4Threads = 256;
constexpr int kFp4Limit = 512;   // threads of a row at most
// Chunks of 16 in a thread's registers at most. In us with 2 / 4 / 8: 128256 x 4096 bf16 nvfp4 294 / 262 / 277,
// mxfp4 221 / 190 / 210, 64128 x 4096 fp32 262 / 214 / 486; through shared memory 3001 x 1111 fp32 6.9 / 8.7.
constexpr int fp4_held(bool whole) { return whole ? 4 : 2; }
constexpr int kFp4Values = 4;    // vectors of 8 per thread, of the values back

// The row's power of two (its byte) and that of its inverse.
struct RowScale {
  uint32_t byte;
  __device__ float value() const { return power_of_byte(byte); }
  __device__ float inverse() const { return inverse_power_of_byte(byte); }
};

// 1 / 6 rounded down, and what is left of it.
constexpr float kSixth = 0x1.555554p-3f, kSixthRest = 0x1.555556p-27f;

// A chunk's codes, eight to a word, and its scale byte (of 16 values, or of 32 with its neighbour's).
// amax: the bits of the block's largest magnitude.
template <int kBf16, int kNv>
__device__ __forceinline__ uint2 quantize_chunk(const Chunk<kBf16>& c, uint32_t amax, RowScale g, uint32_t& byte) {
  float v[16];
  c.widen(v);
  const bool finite = amax < kInfBits;
  if constexpr (kNv) {
    // Powers of two do not round, so v r / g is (v / g) r. In rows so small or so large (below 2^-95, from 2^97 on)
    // that a factor leaves the normal numbers, v is divided by g first, and the largest magnitude in every row: what
    // that takes out of the normal numbers is far below every tie.
    const bool apart = g.byte - 32u > 191u;
    const float a = __uint_as_float(amax) * g.inverse();
    const float sixth = fmaf(a, kSixth, a * kSixthRest);
    byte = finite ? e4m3x2(sixth, 0.f) & 0xFFu : 0x7Fu;
    float s, none;
    widen_e4m3x2(finite ? byte : 0u, s, none);
    // 1 / s = r + rest: the approximate reciprocal, which is off by 2^-23 of it at most, two units lower, so that
    // the rest is not negative and -0 stays -0
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = s > 0.f ? __uint_as_float(__float_as_uint(r) - 2u) : 0.f;
    float rest = fmaf(-s, r, 1.f) * r;
    if (apart) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= g.inverse();
    } else {
      r *= g.inverse();
      rest *= g.inverse();
    }
    const uint64_t rs = pair(r, r), rests = pair(rest, rest);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const uint64_t two = pair(v[e], v[e + 1]);
      split(fma2(two, rs, mul2(two, rests)), v[e], v[e + 1]);
    }
  } else {
    byte = power_scale_byte<2, 0x400000u>(amax);
    const float inv = finite ? inverse_power_of_byte(byte) : 0.f;
    const uint64_t by = pair(inv, inv);
#pragma unroll
    for (int e = 0; e < 16; e += 2) split(mul2(pair(v[e], v[e + 1]), by), v[e], v[e + 1]);
  }
  const float(&lo)[8] = *reinterpret_cast<const float(*)[8]>(v);
  const float(&hi)[8] = *reinterpret_cast<const float(*)[8]>(v + 8);
  return finite ? make_uint2(e2m1x8(lo), e2m1x8(hi)) : make_uint2(0, 0);
}

// Rows up to the next multiple of 128: those past N have scales alone, 0. R threads a row; kHeld: chunks of
// it in a thread's registers; 0: read twice.
template <int kBf16, int kNv, int kWhole, int kHeld>
__global__ void __launch_bounds__(kFp4Limit)
    quantize_fp4_kernel(const void* x, int64_t ldx, int N, int D, uint8_t* codes, uint8_t* scales,
                        float* row_scales, int R) {
  __shared__ uint32_t s_max[kFp4Limit / 32];
  __shared__ float s_stage[kWhole ? 1 : kFp4Limit / 32][kWhole ? 1 : kWarpStage<16>];
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kLanes = kNv ? 1 : 2;   // of a block
  start_next_launch();   // (flce_fp4_gemm.cu's)
  const int t = static_cast<int>(threadIdx.x) % R, warp = static_cast<int>(threadIdx.x) >> 5;
  float* const stage = s_stage[kWhole ? 0 : warp];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / R) + threadIdx.x / R;
  const bool live = row < N;
  const uint8_t* const from = static_cast<const uint8_t*>(x) + row * ldx * kElt;
  const int width = live ? D : 0;
  const int chunks = static_cast<int>(fp4_stages(D)) * (kFp4Stage / 16);
  // where rows are read twice: whole warps go on together, as they load and shuffle together (chunks come in 16s)
  [[maybe_unused]] const int padded = (chunks + R - 1) / R * R;
  const int code_bytes = static_cast<int>(fp4_code_bytes(D));
  // a block's largest magnitude; the row's over its finite values
  auto block_max = [&](const Chunk<kBf16>& c) { return largest_of_lanes<kLanes>(c.largest()); };
  auto row_max = [&](const Chunk<kBf16>& c, uint32_t block, uint32_t m) {
    if (block < kInfBits) return max(m, block);
    float v[16];
    c.widen(v);
#pragma unroll
    for (int e = 0; e < 16; ++e) m = magnitude(v[e]) < kInfBits ? max(m, magnitude(v[e])) : m;
    return m;
  };
  Chunk<kBf16> held[kHeld > 0 ? kHeld : 1];
  uint32_t amax[kHeld > 0 ? kHeld : 1];
  if constexpr (kHeld > 0) {
    load_chunks<kBf16, kWhole>(from, t, R, width, stage, held);
#pragma unroll
    for (int k = 0; k < kHeld; ++k) amax[k] = block_max(held[k]);
  }
  RowScale g{127u};
  if constexpr (kNv) {
    uint32_t m = 0;
    if constexpr (kHeld > 0) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) m = row_max(held[k], amax[k], m);
    } else {
      for (int i = t; i < padded; i += R) {
        Chunk<kBf16> c[1];
        load_chunks<kBf16, kWhole>(from, i, 0, width, stage, c);
        m = row_max(c[0], block_max(c[0]), m);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (R > 32) {
      const int per = R >> 5;
      if ((threadIdx.x & 31) == 0) s_max[warp] = m;
      __syncthreads();
      for (int w = 0; w < per; ++w) m = max(m, s_max[warp / per * per + w]);
    }
    const uint32_t byte = power_scale_byte<11, 0x280000u>(m);
    g.byte = m == 0 ? 127u : byte < 1u ? 1u : byte;
    if (t == 0 && live) row_scales[row] = g.value();
  }
  auto put = [&](int i, const Chunk<kBf16>& c, uint32_t block) {
    uint32_t byte;
    const uint2 code = quantize_chunk<kBf16, kNv>(c, block, g, byte);
    // the bytes of four neighbouring blocks, in the first of their lanes (a block behind the row, whose
    // largest is 0, has the byte 0 too)
    uint32_t w = byte << (8 * ((threadIdx.x / kLanes) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, kLanes);
    w |= __shfl_xor_sync(0xffffffffu, w, 2 * kLanes);
    if (i >= chunks) return;
    if (live && i * 8 < code_bytes) *reinterpret_cast<uint2*>(codes + row * code_bytes + i * 8) = code;
    if (t % (4 * kLanes) == 0)
      *reinterpret_cast<uint32_t*>(scales + fp4_scale_at(row, i / (4 * kLanes), D, kNv)) = w;
  };
  if constexpr (kHeld > 0) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) put(t + k * R, held[k], amax[k]);
  } else {
    for (int i = t; i < padded; i += R) {
      Chunk<kBf16> c[1];
      load_chunks<kBf16, kWhole>(from, i, 0, width, stage, c);
      put(i, c[0], block_max(c[0]));
    }
  }
}

template <int kBf16, int kNv, int kWhole>
__global__ void __launch_bounds__(kFp4Threads)
    dequantize_fp4_kernel(const uint8_t* codes, const uint8_t* scales, const float* row_scales, int N, int D,
                          void* x, int64_t ldx, int X) {
  __shared__ float s_stage[kWhole ? 1 : kFp4Threads / 32][kWhole ? 1 : kWarpStage<8>];
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kBlock = fp4_block(kNv);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kFp4Threads / X) + threadIdx.x / X;
  if (row >= N) return;   // whole warps: X is at least 32
  const int t = static_cast<int>(threadIdx.x) % X;
  uint8_t* const to = static_cast<uint8_t*>(x) + row * ldx * kElt;
  const float row_scale = kNv ? row_scales[row] : 1.f;
  const int first = static_cast<int>(blockIdx.y) * X * kFp4Values + t;
  uint32_t c[kFp4Values] = {}, byte[kFp4Values] = {};
#pragma unroll
  for (int k = 0; k < kFp4Values; ++k) {
    const int i = first + k * X;
    if (i * 8 < D) {
      const int block = i * 8 / kBlock;
      c[k] = *reinterpret_cast<const uint32_t*>(codes + row * fp4_code_bytes(D) + i * 4);
      byte[k] = scales[fp4_scale_at(row, block / 4, D, kNv) + block % 4];
    }
  }
#pragma unroll
  for (int k = 0; k < kFp4Values; ++k) {
    const int i = first + k * X;
    if ((i - (t & 31)) * 8 >= D) break;
    float s, none;
    if (kNv) widen_e4m3x2(byte[k], s, none);
    else s = power_of_byte(byte[k]);
    float v[8];
    widen_e2m1x8(c[k], v);
    const uint64_t by = pair(s, s), rows = pair(row_scale, row_scale);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint64_t two = mul2(pair(v[e], v[e + 1]), by);
      split(kNv ? mul2(two, rows) : two, v[e], v[e + 1]);
    }
    if constexpr (!kWhole) {
      store_staged<kBf16, 8>(to, (i - (t & 31)) * 8, D, s_stage[threadIdx.x >> 5], v);
    } else if (i * 8 + 8 <= D) {
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
                                uint8_t* scales, float* row_scales, cudaStream_t stream) {
  const int chunks = static_cast<int>(fp4_stages(D)) * (kFp4Stage / 16);
  const int64_t rows = (static_cast<int64_t>(N) + kFp4RowTile - 1) / kFp4RowTile * kFp4RowTile;
  const bool whole = whole_vectors(x, bf16, ldx);
  const int R = threads_of_row(N, chunks, fp4_held(whole), 32, kFp4Limit);
  const int block = R < kFp4Threads ? kFp4Threads : R;
  const unsigned grid = static_cast<unsigned>((rows * R + block - 1) / block);
  return with_flags(bf16 != 0, nv != 0, whole, [&](auto b, auto n, auto w) {
    auto go = [&](auto kern) {
      kern<<<grid, block, 0, stream>>>(x, ldx, N, D, codes, scales, row_scales, R);
      return cudaGetLastError();
    };
    const int per = (chunks + R - 1) / R;
    if (per <= 1) return go(quantize_fp4_kernel<b(), n(), w(), 1>);
    if (per <= 2) return go(quantize_fp4_kernel<b(), n(), w(), 2>);
    if constexpr (fp4_held(w()) >= 4)
      if (per <= 4) return go(quantize_fp4_kernel<b(), n(), w(), 4>);
    return go(quantize_fp4_kernel<b(), n(), w(), 0>);
  });
}

cudaError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* row_scales, int N,
                                  int D, int nv, void* x, int bf16, int64_t ldx, cudaStream_t stream) {
  const int nvec = (D + 7) / 8;
  const int X = threads_of_row(N, nvec, kFp4Values, 32, kFp4Threads);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(N) * X + kFp4Threads - 1) / kFp4Threads),
                  static_cast<unsigned>((nvec + X * kFp4Values - 1) / (X * kFp4Values)));
  return with_flags(bf16 != 0, nv != 0, whole_vectors(x, bf16, ldx), [&](auto b, auto n, auto w) {
    dequantize_fp4_kernel<b(), n(), w()><<<grid, kFp4Threads, 0, stream>>>(codes, scales, row_scales, N, D, x, ldx, X);
    return cudaGetLastError();
  });
}

}  // namespace flce
