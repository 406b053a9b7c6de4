// Activations in 8 bits: E4M3 codes with a power-of-two scale for each 32 values of a row, and
// back.
//
// Rows that allow 16-byte accesses: a thread has 8 values, four neighbours a block, whose
// largest magnitude meets over two shuffles. Other rows: a lane has one value, a warp a block, so
// that accesses of 2 or 4 bytes stay side by side. Each thread has kAtOnce vectors (or blocks) in
// flight.
//
// Bound by the bytes: D + D / 32 written or read for 2 D or 4 D.
#include <cstdint>

#include "flce_blocks.cuh"
#include "flce_norm.cuh"

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

// X threads per row, from vector first on; x 16-byte aligned rows.
template <int kBf16>
__global__ void __launch_bounds__(kPackThreads)
    pack_kernel(const void* x, int64_t ldx, int N, int D, uint8_t* packed, int X) {
  constexpr int kElt = kBf16 ? 2 : 4;
  using In = Param<kBf16, 8>;
  const int row = blockIdx.x * (kPackThreads / X) + static_cast<int>(threadIdx.x) / X;
  const int t = static_cast<int>(threadIdx.x) % X;
  const bool live = row < N;   // whole warps go on together, for the shuffles
  const uint8_t* const from = static_cast<const uint8_t*>(x) + row * ldx * kElt;
  uint8_t* const record = packed + row * packed_record(D);
  const int nvec = static_cast<int>(packed_codes(D)) / 8;
  const int first = static_cast<int>(blockIdx.y) * X * kAtOnce + t;
  In in[kAtOnce];
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int i = first + k * X;
    in[k].load_if(from, i * 8, live && i * 8 + 8 <= D);
  }
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int i = first + k * X;
    float v[8];
    in[k].widen(v);
    if (live && i * 8 < D && i * 8 + 8 > D) {   // the vector in which the row ends
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i * 8 + e < D ? load_as_f32(from, i * 8 + e, kBf16) : 0.f;
    }
    const uint32_t byte = e4m3_scale_byte(largest_of_lanes<4>(largest_bits(v)));
    if (live && i < nvec) {
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
  if (live && blockIdx.y == 0) pad_scales(record, D, t, X);
}

// A warp per row piece: kAtOnce blocks, a value per lane.
template <int kBf16>
__global__ void __launch_bounds__(kPackThreads)
    pack_narrow_kernel(const void* x, int64_t ldx, int N, int D, uint8_t* packed, int pieces) {
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(warp / pieces);
  if (row >= N) return;
  const int piece = static_cast<int>(warp % pieces);
  const int blocks = static_cast<int>(packed_codes(D)) / kPackBlock;
  uint8_t* const record = packed + row * packed_record(D);
  float v[kAtOnce];
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int i = (piece * kAtOnce + k) * 32 + lane;
    v[k] = i < D ? load_as_f32(x, row * ldx + i, kBf16) : 0.f;
  }
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int block = piece * kAtOnce + k;
    if (block >= blocks) break;
    const uint32_t byte = e4m3_scale_byte(__reduce_max_sync(0xffffffffu, magnitude(v[k])));
    const uint32_t code = byte == 255u ? (block * 32 + lane < D ? 0x7Fu : 0u) : e4m3x2(v[k] * inverse_power_of_byte(byte), 0.f) & 0xFFu;
    record[block * 32 + lane] = static_cast<uint8_t>(code);
    if (lane == 0) record[packed_codes(D) + block] = static_cast<uint8_t>(byte);
  }
  if (piece == 0) pad_scales(record, D, lane, 32);
}

template <int kBf16>
__global__ void __launch_bounds__(kPackThreads)
    unpack_kernel(const uint8_t* packed, int N, int D, void* x, int64_t ldx, int X) {
  constexpr int kElt = kBf16 ? 2 : 4;
  const int row = blockIdx.x * (kPackThreads / X) + static_cast<int>(threadIdx.x) / X;
  if (row >= N) return;
  const int t = static_cast<int>(threadIdx.x) % X;
  const uint8_t* const record = packed + row * packed_record(D);
  uint8_t* const to = static_cast<uint8_t*>(x) + row * ldx * kElt;
  const int first = static_cast<int>(blockIdx.y) * X * kAtOnce + t;
  uint2 codes[kAtOnce];
  uint32_t byte[kAtOnce];
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
    if (i * 8 >= D) break;
    const float s = power_of_byte(byte[k]);
    float v[8];
    widen_e4m3x2(codes[k].x, v[0], v[1]);
    widen_e4m3x2(codes[k].x >> 16, v[2], v[3]);
    widen_e4m3x2(codes[k].y, v[4], v[5]);
    widen_e4m3x2(codes[k].y >> 16, v[6], v[7]);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= s;
    if (i * 8 + 8 <= D) {
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

template <int kBf16>
__global__ void __launch_bounds__(kPackThreads)
    unpack_narrow_kernel(const uint8_t* packed, int N, int D, void* x, int64_t ldx, int pieces) {
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(warp / pieces);
  if (row >= N) return;
  const int piece = static_cast<int>(warp % pieces);
  const uint8_t* const record = packed + row * packed_record(D);
  uint32_t code[kAtOnce], byte[kAtOnce];
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int block = piece * kAtOnce + k;
    if (block * 32 + lane < D) {
      code[k] = record[block * 32 + lane];
      byte[k] = record[packed_codes(D) + block];
    }
  }
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int i = (piece * kAtOnce + k) * 32 + lane;
    if (i >= D) break;
    float v, none;
    widen_e4m3x2(code[k], v, none);
    store_from_f32(x, row * ldx + i, v * power_of_byte(byte[k]), kBf16);
  }
}

bool whole_vectors(const void* x, int bf16, int64_t ldx) {
  return reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * (bf16 ? 2 : 4) % 16 == 0;
}

// f(grid, X) for rows of nvec vectors, X threads a row (whole groups of four).
template <typename F>
cudaError_t row_grid(int N, int nvec, F&& f) {
  int X = 4;
  while (X < kPackThreads && X < nvec) X *= 2;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(N) * X + kPackThreads - 1) / kPackThreads),
                  static_cast<unsigned>((nvec + X * kAtOnce - 1) / (X * kAtOnce)));
  f(grid, X);
  return cudaGetLastError();
}

// f(grid, pieces): a warp for each kAtOnce blocks of a row.
template <typename F>
cudaError_t warp_grid(int N, int D, F&& f) {
  const int pieces = (D + 32 * kAtOnce - 1) / (32 * kAtOnce);
  const int64_t threads = static_cast<int64_t>(N) * pieces * 32;
  f(static_cast<unsigned>((threads + kPackThreads - 1) / kPackThreads), pieces);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pack_e4m3(const void* x, int bf16, int64_t ldx, int N, int D, uint8_t* packed,
                             cudaStream_t stream) {
  if (whole_vectors(x, bf16, ldx))
    return row_grid(N, static_cast<int>(packed_codes(D)) / 8, [&](dim3 grid, int X) {
      if (bf16) pack_kernel<1><<<grid, kPackThreads, 0, stream>>>(x, ldx, N, D, packed, X);
      else pack_kernel<0><<<grid, kPackThreads, 0, stream>>>(x, ldx, N, D, packed, X);
    });
  return warp_grid(N, D, [&](unsigned grid, int pieces) {
    if (bf16) pack_narrow_kernel<1><<<grid, kPackThreads, 0, stream>>>(x, ldx, N, D, packed, pieces);
    else pack_narrow_kernel<0><<<grid, kPackThreads, 0, stream>>>(x, ldx, N, D, packed, pieces);
  });
}

cudaError_t launch_unpack_e4m3(const uint8_t* packed, int N, int D, void* x, int bf16, int64_t ldx,
                               cudaStream_t stream) {
  if (whole_vectors(x, bf16, ldx))
    return row_grid(N, (D + 7) / 8, [&](dim3 grid, int X) {
      if (bf16) unpack_kernel<1><<<grid, kPackThreads, 0, stream>>>(packed, N, D, x, ldx, X);
      else unpack_kernel<0><<<grid, kPackThreads, 0, stream>>>(packed, N, D, x, ldx, X);
    });
  return warp_grid(N, D, [&](unsigned grid, int pieces) {
    if (bf16) unpack_narrow_kernel<1><<<grid, kPackThreads, 0, stream>>>(packed, N, D, x, ldx, pieces);
    else unpack_narrow_kernel<0><<<grid, kPackThreads, 0, stream>>>(packed, N, D, x, ldx, pieces);
  });
}

}  // namespace flce
