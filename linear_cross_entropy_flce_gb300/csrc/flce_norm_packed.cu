// Layer norm, forward, that leaves its input in 8 bits as well:
//   y = (x - mean) rstd weight + bias, and x in E4M3 with a power of two for each 32 values.
//
// A group of R threads holds a row in registers as it was loaded, 16 neighbouring values a chunk, up to
// two chunks each, and widens it again for each use: the sum, the variance (from centred values), the codes,
// the output. Rows that do not allow 16-byte accesses come and go through shared memory, a warp's 512
// values at a time. Which calls come here is decided, with figures, in flce_norm.cu.
//
// Bound by instructions and their latency: 16384 x 1024 bf16 17.1 us, 4000 x 4096 18.9, of which the bytes are 12.6
// and 12.3 (8192 x 4096 36 us; 50 with registers for 16 warps an SM instead of 32, 40.8 with two rows of a chunk
// a thread).
#include <cstdint>

#include "flce_blocks.cuh"
#include "flce_norm_stream.cuh"

namespace flce {

namespace {

constexpr int kNormPackThreads = 256;
constexpr int kNormPackLimit = 512;   // threads of a row at most
constexpr int kNormPackHeld = 2;      // chunks in a thread's registers at most

// 16 values of weight or bias (or `none` without one) from element i on; what is behind D is not read.
template <int kWbf16>
__device__ __forceinline__ void load_param16(const void* p, int wide, int i, int D, float none, float (&v)[16]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = none;
  } else if (wide && i + 16 <= D) {
    Chunk<kWbf16> c;
    c.load_if(static_cast<const uint8_t*>(p), i / 16, true);
    c.widen(v);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = i + e < D ? load_as_f32(p, i + e, kWbf16) : none;
  }
}

template <int kBf16, int kWbf16, int kWhole, int kHeld>
__global__ void __launch_bounds__(kNormPackLimit, 2)
    norm_pack_kernel(const void* x, int64_t ldx, const void* weight, const void* bias, int wide_params, int N, int D,
                     float eps, void* y, int64_t ldy, float* mean_out, float* rstd_out, uint8_t* packed, int R) {
  __shared__ float2 s_sum[kNormPackLimit / 32], s_sq[kNormPackLimit / 32];
  __shared__ float s_stage[kWhole ? 1 : kNormPackLimit / 32][kWhole ? 1 : kWarpStage<16>];
  constexpr int kElt = kBf16 ? 2 : 4;
  const int group = static_cast<int>(threadIdx.x) / R, t = static_cast<int>(threadIdx.x) % R;
  float* const stage = s_stage[kWhole ? 0 : threadIdx.x >> 5];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / R) + group;
  const bool live = row < N;
  const int width = live ? D : 0;
  const uint8_t* const from = static_cast<const uint8_t*>(x) + row * ldx * kElt;
  const float inv_d = 1.f / static_cast<float>(D);
  Chunk<kBf16> c[kHeld];
  load_chunks<kBf16, kWhole>(from, t, R, width, stage, c);
  uint64_t two = pair(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    float v[16];
    c[k].widen(v);
#pragma unroll
    for (int e = 0; e < 16; e += 2) two = add2(two, pair(v[e], v[e + 1]));
  }
  float part, other;
  split(two, part, other);
  part += other;
  const float mean = stream_sum2(make_float2(part, 0.f), group, R, s_sum).x * inv_d;
  // the codes, while the others arrive
  uint8_t* const record = packed + row * packed_record(D);
  const int codes = static_cast<int>(packed_codes(D));
  const uint64_t less = pair(-mean, -mean);
  two = pair(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = (t + k * R) * 16;
    float v[16];
    c[k].widen(v);
    const uint32_t byte = e4m3_scale_byte(largest_of_lanes<2>(c[k].largest()));
    if (live && i < codes) {
      uint4 q;
      if (byte != 255u) {
        const float inv = inverse_power_of_byte(byte);
        q = make_uint4(e4m3x4(v, inv), e4m3x4(v + 4, inv), e4m3x4(v + 8, inv), e4m3x4(v + 12, inv));
      } else {   // NaN, but for what is behind the row
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (e % 4 == 0) w[e / 4] = 0;
          if (i + e < D) w[e / 4] |= 0x7Fu << (e % 4 * 8);
        }
        q = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(record + i) = q;
      if (i % kPackBlock == 0) record[codes + i / kPackBlock] = static_cast<uint8_t>(byte);
    }
    if (i + 16 <= D) {
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const uint64_t d = add2(pair(v[e], v[e + 1]), less);
        two = fma2(d, d, two);
      }
    } else {
      split(two, part, other);
#pragma unroll
      for (int e = 0; e < 16; ++e) part = i + e < D ? fmaf(v[e] - mean, v[e] - mean, part) : part;
      two = pair(part, other);
    }
  }
  split(two, part, other);
  part += other;
  if (live)
    for (int i = codes / kPackBlock * 33 + t; i < packed_record(D); i += R) record[i] = 0;
  // rsqrtf is off by 2 units of its last place at most, below the sums' own rounding
  const float rstd = rsqrtf(stream_sum2(make_float2(part, 0.f), group, R, s_sq).x * inv_d + eps);
  uint8_t* const to = static_cast<uint8_t*>(y) + row * ldy * kElt;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = (t + k * R) * 16;
    if (kWhole && i >= D) break;
    float v[16], w[16], b[16];
    c[k].widen(v);
    load_param16<kWbf16>(weight, wide_params, i, D, 1.f, w);
    load_param16<kWbf16>(bias, wide_params, i, D, 0.f, b);
#pragma unroll
    for (int e = 0; e < 16; e += 2)
      split(fma2(mul2(add2(pair(v[e], v[e + 1]), less), pair(rstd, rstd)), pair(w[e], w[e + 1]), pair(b[e], b[e + 1])),
            v[e], v[e + 1]);
    if constexpr (!kWhole) {
      store_staged<kBf16, 16>(to, i - (t & 31) * 16, width, stage, v);
    } else if (live) {
      if (i + 16 <= D) {
        Chunk<kBf16> out;
        out.narrow(v);
#pragma unroll
        for (int q = 0; q < (kBf16 ? 2 : 4); ++q) reinterpret_cast<uint4*>(to + i * kElt)[q] = out.w[q];
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (i + e < D) store_from_f32(to, i + e, v[e], kBf16);
      }
    }
  }
  if (t == 0 && live) {
    if (mean_out != nullptr) mean_out[row] = mean;
    if (rstd_out != nullptr) rstd_out[row] = rstd;
  }
}

}  // namespace

cudaError_t launch_norm_pack(const void* x, int bf16, int64_t ldx, const void* weight, const void* bias,
                             int wbf16, int N, int D, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                             uint8_t* packed, cudaStream_t stream) {
  const int chunks = static_cast<int>(packed_codes(D)) / 16;
  const int R = threads_of_row(N, chunks, kNormPackHeld, 32, kNormPackLimit);
  const int per = (chunks + R - 1) / R;
  if (per > kNormPackHeld) return cudaErrorNotSupported;
  const int block = R < kNormPackThreads ? kNormPackThreads : R, rows = block / R;
  const bool whole = whole_vectors(x, bf16, ldx) && whole_vectors(y, bf16, ldy);
  const int wide = whole_vectors(weight, 0, 0) && whole_vectors(bias, 0, 0);
  return with_stream_types(bf16, wbf16, whole, [&](auto b, auto wb, auto w) {
    auto go = [&](auto kern) {
      kern<<<static_cast<unsigned>((N + rows - 1) / rows), block, 0, stream>>>(
          x, ldx, weight, bias, wide, N, D, eps, y, ldy, mean, rstd, packed, R);
      return cudaGetLastError();
    };
    if (per <= 1) return go(norm_pack_kernel<b(), wb(), w(), 1>);
    return go(norm_pack_kernel<b(), wb(), w(), kNormPackHeld>);
  });
}

}  // namespace flce
