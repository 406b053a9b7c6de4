// Activations in 8 bits: E4M3 codes with a power-of-two scale for each 32 values of a row, and
// back.
//
// A thread has 8 neighbouring values, four neighbours a block, whose largest magnitude meets over two
// shuffles; rows that do not allow 16-byte accesses go through shared memory, a warp's 256 values
// at a time. Each thread has kAtOnce vectors in flight.
//
// Bound by the bytes, D + D / 32 written or read for 2 D or 4 D, and the instructions beside them: 16384 x 8192
// bf16 65 us packed and 59 unpacked (0.94 and 1.02 of the copy rate), 8192 x 4096 18.0 and 14.2, 4000 x 4096 fp32
// 13.1 and 18.0, 3001 x 1111 fp32 5.9 and 4.2, 1 x 4096 1.9 and 1.8. As many threads a row as have kAtOnce vectors
// each: with a thread for each vector 8192 x 4096 took 26.8 and 17.4.
#include <cstdint>

#include "flce_blocks.cuh"

namespace flce {

namespace {

constexpr int kPackThreads = 256;
constexpr int kAtOnce = 4;

// The zeros behind a row's scale bytes, by X threads.
__device__ __forceinline__ void pad_scales(uint8_t* record, int D, int t, int X) {
  const int blocks = static_cast<int>(packed_codes(D)) / kPackBlock;
  const int end = static_cast<int>(packed_record(D) - packed_codes(D));
  for (int b = blocks + t; b < end; b += X) record[packed_codes(D) + b] = 0;
}

// X threads per row. kWhole: 16-byte accesses.
template <int kBf16, int kWhole>
__global__ void __launch_bounds__(kPackThreads)
    pack_kernel(const void* x, int64_t ldx, int N, int D, uint8_t* packed, int X) {
  __shared__ float s_stage[kWhole ? 1 : kPackThreads / 32][kWhole ? 1 : kWarpStage<8>];
  constexpr int kElt = kBf16 ? 2 : 4;
  using In = Param<kBf16, 8>;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kPackThreads / X) + threadIdx.x / X;
  const int t = static_cast<int>(threadIdx.x) % X;
  const int width = row < N ? D : 0;   // whole warps go on together, for the shuffles
  const uint8_t* const from = static_cast<const uint8_t*>(x) + row * ldx * kElt;
  uint8_t* const record = packed + row * packed_record(D);
  const int nvec = static_cast<int>(packed_codes(D)) / 8;
  const int first = static_cast<int>(blockIdx.y) * X * kAtOnce + t;
  [[maybe_unused]] In in[kAtOnce];
  if constexpr (kWhole) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) in[k].load_if(from, (first + k * X) * 8, (first + k * X) * 8 + 8 <= width);
  }
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int i = first + k * X;
    if (i - (t & 31) >= nvec) break;   // the warp's first (X is at least 32)
    float v[8];
    if constexpr (kWhole) {
      in[k].widen(v);
      if (i * 8 < width && i * 8 + 8 > width) {   // the vector in which the row ends
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = i * 8 + e < width ? load_as_f32(from, i * 8 + e, kBf16) : 0.f;
      }
    } else {
      float apart[8];   // (all vectors' loads first, in 32 registers, took 73 us instead of 58 for 16000 x 4001 bf16)
      load_apart<kBf16, 8>(from, (i - (t & 31)) * 8, width, apart);
      to_neighbours(apart, s_stage[threadIdx.x >> 5], v);
    }
    const uint32_t byte = e4m3_scale_byte(largest_of_lanes<4>(largest_bits(v)));
    if (row < N && i < nvec) {
      const float inv = byte == 255u ? 0.f : inverse_power_of_byte(byte);
      uint2 codes = make_uint2(e4m3x4(v, inv), e4m3x4(v + 4, inv));
      if (byte == 255u) {   // NaN, but for what is behind the row
        const int n = D - i * 8;
        const uint64_t all = n <= 0 ? 0 : n >= 8 ? ~0ull : (1ull << (8 * n)) - 1;
        codes = make_uint2(0x7F7F7F7Fu & static_cast<uint32_t>(all), 0x7F7F7F7Fu & static_cast<uint32_t>(all >> 32));
      }
      *reinterpret_cast<uint2*>(record + i * 8) = codes;
      if (i % 4 == 0) record[packed_codes(D) + i / 4] = static_cast<uint8_t>(byte);
    }
  }
  if (row < N && blockIdx.y == 0) pad_scales(record, D, t, X);
}

template <int kBf16, int kWhole>
__global__ void __launch_bounds__(kPackThreads)
    unpack_kernel(const uint8_t* packed, int N, int D, void* x, int64_t ldx, int X) {
  __shared__ float s_stage[kWhole ? 1 : kPackThreads / 32][kWhole ? 1 : kWarpStage<8>];
  constexpr int kElt = kBf16 ? 2 : 4;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kPackThreads / X) + threadIdx.x / X;
  if (row >= N) return;   // whole warps: X is at least 32
  const int t = static_cast<int>(threadIdx.x) % X;
  const uint8_t* const record = packed + row * packed_record(D);
  uint8_t* const to = static_cast<uint8_t*>(x) + row * ldx * kElt;
  const int first = static_cast<int>(blockIdx.y) * X * kAtOnce + t;
  uint2 codes[kAtOnce] = {};
  uint32_t byte[kAtOnce] = {};
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int i = first + k * X;
    if (i * 8 < D) {
      codes[k] = *reinterpret_cast<const uint2*>(record + i * 8);
      byte[k] = record[packed_codes(D) + i / 4];
    }
  }
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int i = first + k * X;
    if ((i - (t & 31)) * 8 >= D) break;
    const float s = power_of_byte(byte[k]);
    float v[8];
    widen_e4m3x2(codes[k].x, v[0], v[1]);
    widen_e4m3x2(codes[k].x >> 16, v[2], v[3]);
    widen_e4m3x2(codes[k].y, v[4], v[5]);
    widen_e4m3x2(codes[k].y >> 16, v[6], v[7]);
    const uint64_t by = pair(s, s);
#pragma unroll
    for (int e = 0; e < 8; e += 2) split(mul2(pair(v[e], v[e + 1]), by), v[e], v[e + 1]);
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

// f(grid, X) for rows of nvec vectors, X threads a row.
template <typename F>
cudaError_t row_grid(int N, int nvec, F&& f) {
  const int X = threads_of_row(N, nvec, kAtOnce, 32, kPackThreads);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(N) * X + kPackThreads - 1) / kPackThreads),
                  static_cast<unsigned>((nvec + X * kAtOnce - 1) / (X * kAtOnce)));
  f(grid, X);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pack_e4m3(const void* x, int bf16, int64_t ldx, int N, int D, uint8_t* packed,
                             cudaStream_t stream) {
  const bool whole = whole_vectors(x, bf16, ldx);
  return row_grid(N, static_cast<int>(packed_codes(D)) / 8, [&](dim3 grid, int X) {
    auto go = [&](auto kern) { kern<<<grid, kPackThreads, 0, stream>>>(x, ldx, N, D, packed, X); };
    if (bf16) whole ? go(pack_kernel<1, 1>) : go(pack_kernel<1, 0>);
    else whole ? go(pack_kernel<0, 1>) : go(pack_kernel<0, 0>);
  });
}

cudaError_t launch_unpack_e4m3(const uint8_t* packed, int N, int D, void* x, int bf16, int64_t ldx,
                               cudaStream_t stream) {
  const bool whole = whole_vectors(x, bf16, ldx);
  return row_grid(N, (D + 7) / 8, [&](dim3 grid, int X) {
    auto go = [&](auto kern) { kern<<<grid, kPackThreads, 0, stream>>>(packed, N, D, x, ldx, X); };
    if (bf16) whole ? go(unpack_kernel<1, 1>) : go(unpack_kernel<1, 0>);
    else whole ? go(unpack_kernel<0, 1>) : go(unpack_kernel<0, 0>);
  });
}

}  // namespace flce
