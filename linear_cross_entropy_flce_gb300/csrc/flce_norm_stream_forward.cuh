// Layer norm of many rows, forward: y = (x - mean) rstd weight + bias.
//
// Rows come through the ring (flce_norm_stream.cuh), two at a time: a thread holds the same
// 64 bytes of columns of both in registers, so that the barriers of a turn and the reads of
// weight and bias (from shared memory) serve two rows. The variance is taken from centred
// values. Once the group has read its rows, the copies of the rows kRing turns ahead start
// into their place, while the variance and the output are still to come.
//
// Bound by instructions and barriers as much as by bytes: 8192 x 4096 bf16 26.7 us (5.0 TB/s
// of rows read and written; one row of a turn 32 us, three turns in the ring 28), 16384 x 8192
// 91 us (5.9 TB/s), 4000 x 4096 fp32 24.7 us (5.3 TB/s). Ragged rows (by the kernel of rows in
// registers in brackets): 3001 x 1111 fp32 10.9 us (17.4), 16384 x 2730 bf16 61 (83), 16000 x
// 4001 bf16 76 (148). A full CTA has 512 threads, as many as 128
// registers each allow.
//
// kPacked: x is left in 8 bits as well (flce_pack.cu's records): whole rows from the registers the row is in;
// ragged rows, whose blocks do not begin with a chunk, from the ring, before it is filled again.
// 16384 x 8192 bf16 115.5 us (5.8 TB/s), 8192 x 4096 33, 4000 x 4096 fp32 29.8, 3001 x 1111 fp32 12.8, 16000 x 4001
// bf16 107. Two values an instruction: it is bound by instructions.
#pragma once

#include <cstdint>

#include "flce_blocks.cuh"
#include "flce_norm_stream.cuh"
#include "flce_norm_stream.h"

namespace flce {

namespace {

constexpr int kForwardBlock = 512;
constexpr int kRing = 2;   // turns of a group in the ring, of two rows each

// VW neighbouring values to a record's codes and, by the first lane of a block's, its scale byte; largest: of the
// block. `there`: element i is before the codes' end.
template <int VW>
__device__ __forceinline__ void pack_values(uint8_t* record, int i, int D, const float (&v)[VW], uint32_t largest,
                                            bool there) {
  if (!there) return;
  const uint32_t byte = e4m3_scale_byte(largest);
  uint32_t codes[VW / 4];
  if (byte != 255u) {
    const float inv = inverse_power_of_byte(byte);
#pragma unroll
    for (int k = 0; k < VW / 4; ++k) codes[k] = e4m3x4(v + 4 * k, inv);
  } else {   // NaN, but for what is behind the row
#pragma unroll
    for (int k = 0; k < VW / 4; ++k) {
      codes[k] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + 4 * k + e < D) codes[k] |= 0x7Fu << (8 * e);
    }
  }
  if constexpr (VW == 8) *reinterpret_cast<uint2*>(record + i) = make_uint2(codes[0], codes[1]);
  else *reinterpret_cast<uint32_t*>(record + i) = codes[0];
  if (i % kPackBlock == 0) record[packed_codes(D) + i / kPackBlock] = static_cast<uint8_t>(byte);
}

template <int kBf16, int kWbf16, int kRagged, int kNv, int kPacked>
__global__ void __launch_bounds__(kForwardBlock, 1)
    norm_stream_kernel(const void* x, int64_t ldx, const void* weight, const void* bias, int N,
                       int D, float eps, void* y, int64_t ldy, float* mean_out, float* rstd_out,
                       uint8_t* packed, int R, int slot_bytes, int apart) {
  constexpr int kElt = kBf16 ? 2 : 4, kWelt = kWbf16 ? 2 : 4, VW = 16 / kElt;
  constexpr int kFetchers = kRagged ? 32 : 1;
  using E = Each<kPacked>;
  using P = Pack<kBf16, VW>;
  using Raw = typename P::Raw;
  using W = Param<kWbf16, VW>;
  extern __shared__ uint4 s_dyn[];
  __shared__ __align__(8) uint64_t s_full[kForwardBlock / 32][kRing];
  __shared__ float2 s_sum[kForwardBlock / 32], s_sq[kForwardBlock / 32];
  const int groups = static_cast<int>(blockDim.x) / R;
  const int group = threadIdx.x / R, t = threadIdx.x % R;
  const float inv_d = 1.f / static_cast<float>(D);
  const RowPlace<kElt, kRagged> place(static_cast<const uint8_t*>(x) + blockIdx.x * ldx * kElt, D);
  const int chunks = place.chunks;
  [[maybe_unused]] const int codes = static_cast<int>(packed_codes(D));
  // [each group's ring, and two rows on their way out][weight][bias]
  const int group_bytes = (kRing + (kRagged && apart ? 1 : 0)) * 2 * slot_bytes;
  uint8_t* const ring = reinterpret_cast<uint8_t*>(s_dyn) + group * group_bytes;
  uint8_t* const staged = ring + kRing * 2 * slot_bytes;
  uint8_t* const s_w = reinterpret_cast<uint8_t*>(s_dyn) + groups * group_bytes;
  uint8_t* const s_b = s_w + (weight != nullptr ? slot_bytes / kElt * kWelt : 0);

  // a turn takes rows `row` and `row + half`; where any will do, the CTA's lie side by side
  const int64_t all = static_cast<int64_t>(gridDim.x) * groups, step = 2 * all;
  const int64_t half = kRagged ? all : 1;
  const int64_t first = kRagged ? blockIdx.x + static_cast<int64_t>(gridDim.x) * group
                                : (static_cast<int64_t>(blockIdx.x) * groups + group) * 2;
  // by the first 32 threads of a group, or its first
  auto fetch = [&](int64_t row, int slot, uint32_t& single) {
    if (row >= N) return;
    const bool two = row + half < N;
    const uint8_t* from = static_cast<const uint8_t*>(x) + row * ldx * kElt;
    uint8_t* const to = ring + slot * 2 * slot_bytes;
    if (t == 0) {
      const uint32_t bar = smem_u32(&s_full[group][slot]);
      mbar_arrive_expect_tx(bar, place.whole_bytes(D) * (two ? 2 : 1));
      place.copy(smem_u32(to), from, D, bar);
      if (two) place.copy(smem_u32(to + slot_bytes), from + half * ldx * kElt, D, bar);
    }
    if (kRagged && row + (t >> 4) * half < N)   // 16 lanes for each row
      single = place.read_single(from + (t >> 4) * half * ldx * kElt, t & 15, D);
  };
  auto land = [&](int slot, uint32_t single) {
    if (kRagged && t < 32)
      place.write_single(ring + (slot * 2 + (t >> 4)) * slot_bytes, t & 15, D, single);
  };
  if (t == 0) {
    for (int k = 0; k < kRing; ++k) mbar_init(smem_u32(&s_full[group][k]), 1);
    fence_mbar_init();
  }
  uint32_t single[kRing] = {};
  if (t < kFetchers) {
#pragma unroll
    for (int k = 0; k < kRing; ++k) fetch(first + k * step, k, single[k]);
  }
  stage_params<kWbf16, VW, kRagged>(weight, s_w, bias, s_b, place.s, chunks, D);
#pragma unroll
  for (int k = 0; k < kRing; ++k) land(k, single[k]);
  __syncthreads();
  const volatile int never = 0;
  uint64_t limit = kStreamWaitNs;
  int slot = 0;
  uint32_t phase = 0;
  for (int64_t row = first; row < N; row += step) {
    float nan = 0.f;   // a copy that never came makes its row NaN
    if (!mbar_wait_bounded(smem_u32(&s_full[group][slot]), phase, limit, &never)) {
      nan = __uint_as_float(0x7FC00000u);
      if (t == 0 && limit != 0) drain_ring(s_full[group], kRing, slot, phase, row, step, N);
      limit = 0;
    }
    const uint8_t* in = ring + slot * 2 * slot_bytes;
    // In the last turn of an odd number, the second half of the slot is old or unset: its
    // values meet no others and are not stored. Elements past the row count as zeros, and as
    // zeros from the mean.
    const bool two = row + half < N;
    auto inside = [&](int k) { return k < kNv - 1 || t + k * R < chunks; };
    if constexpr (kPacked && kRagged) {   // each vector of the row put together from two chunks
      const int shift = place.s * kElt, q = shift >> 2, bits = (shift & 3) * 8;
      for (int c = t; (c - (t & 31)) * VW < codes; c += R) {
        const int i = c * VW;
        float of[2][VW];
        uint32_t largest[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* const from = in + r * slot_bytes;
          P::widen(of_two_chunks(P::load_if(from, c * VW, c < chunks),
                                 P::load_if(from, (c + 1) * VW, c + 1 < chunks), q, bits), of[r]);
          if (i + VW > D) {
#pragma unroll
            for (int e = 0; e < VW; ++e) of[r][e] = i + e < D ? of[r][e] : 0.f;
          }
          largest[r] = largest_bits(of[r]);
        }
#pragma unroll
        for (int o = 1; o < kPackBlock / VW; o <<= 1) {
#pragma unroll
          for (int r = 0; r < 2; ++r) largest[r] = max(largest[r], __shfl_xor_sync(0xffffffffu, largest[r], o));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
          pack_values<VW>(packed + (row + r * half) * packed_record(D), i, D, of[r], largest[r],
                          i < codes && (r == 0 || two));
      }
    }
    Raw raw[2][kNv];
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      raw[0][k] = P::load_if(in, (t + k * R) * VW, inside(k));
      raw[1][k] = P::load_if(in + slot_bytes, (t + k * R) * VW, inside(k));
    }
    float v[2][kNv][VW], part[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float acc[VW];
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        P::widen(raw[r][k], v[r][k]);
        place.mask(v[r][k], t + k * R, D);
        if (k == 0) {
#pragma unroll
          for (int e = 0; e < VW; ++e) acc[e] = v[r][0][e];
        } else {
          E::add(acc, v[r][k]);
        }
      }
      part[r] = sum_n(acc);
    }
    if constexpr (kPacked && !kRagged) {   // all blocks' shuffles side by side
      uint32_t largest[2][kNv];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
          if constexpr (kBf16) largest[r][k] = largest_bits_bf16<VW / 2>(reinterpret_cast<const uint32_t*>(&raw[r][k]));
          else largest[r][k] = largest_bits(v[r][k]);
        }
      }
#pragma unroll
      for (int o = 1; o < kPackBlock / VW; o <<= 1) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int k = 0; k < kNv; ++k)
            largest[r][k] = max(largest[r][k], __shfl_xor_sync(0xffffffffu, largest[r][k], o));
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int k = 0; k < kNv; ++k) {
          const int i = (t + k * R) * VW;
          pack_values<VW>(packed + (row + r * half) * packed_record(D), i, D, v[r][k], largest[r][k],
                          i < codes && (r == 0 || two));
        }
      }
    }
    const float2 sum = stream_sum2(make_float2(part[0] + nan, part[1] + nan), group, R, s_sum);
    const float mean[2] = {sum.x * inv_d, sum.y * inv_d};
    if (R == 32) __syncwarp();
    if (t < kFetchers && limit != 0) {   // everyone has read the slot; those reads come before the copies' writes
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      fetch(row + kRing * step, slot, single[0]);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float acc[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) acc[e] = 0.f;
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        const float m = inside(k) ? mean[r] : 0.f;
        if constexpr (kPacked) {
          const uint64_t less = pair(-m, -m);
#pragma unroll
          for (int e = 0; e < VW; e += 2)
            split(add2(pair(v[r][k][e], v[r][k][e + 1]), less), v[r][k][e], v[r][k][e + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < VW; ++e) v[r][k][e] -= m;
        }
        place.mask(v[r][k], t + k * R, D);
        E::fma(acc, v[r][k], v[r][k], acc);
      }
      part[r] = sum_n(acc);
    }
    // rsqrtf is off by 2 units of its last place at most, below the sums' own rounding
    const float2 sq = stream_sum2(make_float2(part[0], part[1]), group, R, s_sq);
    const float rstd[2] = {rsqrtf(sq.x * inv_d + eps), rsqrtf(sq.y * inv_d + eps)};
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      if (!inside(k)) break;
      const int c = t + k * R;
      float w[VW], b[VW];
      W p;
      if (weight != nullptr) {
        p.load(s_w, c * VW, 1.f);
        p.widen(w);
      }
      if (bias != nullptr) {
        p.load(s_b, c * VW, 0.f);
        p.widen(b);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (kPacked) {
          if (weight == nullptr) {
#pragma unroll
            for (int e = 0; e < VW; ++e) w[e] = 1.f;
          }
          if (bias == nullptr) {
#pragma unroll
            for (int e = 0; e < VW; ++e) b[e] = 0.f;
          }
          const uint64_t by = pair(rstd[r], rstd[r]);
#pragma unroll
          for (int e = 0; e < VW; e += 2)
            split(fma2(mul2(pair(v[r][k][e], v[r][k][e + 1]), by), pair(w[e], w[e + 1]), pair(b[e], b[e + 1])),
                  v[r][k][e], v[r][k][e + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            float& o = v[r][k][e];
            o *= rstd[r];
            if (weight != nullptr) o = bias != nullptr ? fmaf(o, w[e], b[e]) : o * w[e];
            else if (bias != nullptr) o += b[e];
          }
        }
        if (kRagged && apart) P::store(staged + r * slot_bytes, c * VW, v[r][k]);
        else if (r == 0 || two) place.template store<kBf16>(y, (row + r * half) * ldy, v[r][k], c, D);
      }
    }
    if (kRagged && apart) {
      group_sync(group, R);
      for (int r = 0; r < 1 + two; ++r)
        place.copy_out(staged + r * slot_bytes,
                       static_cast<uint8_t*>(y) + (row + r * half) * ldy * kElt, D, t, R);
    }
    if constexpr (kPacked) {   // the zeros behind the scales
      for (int r = 0; r < 1 + two; ++r)
        for (int i = codes / kPackBlock * 33 + t; i < packed_record(D); i += R)
          packed[(row + r * half) * packed_record(D) + i] = 0;
    }
    if (t == 0)
      for (int r = 0; r < 1 + two; ++r) {
        if (mean_out != nullptr) mean_out[row + r * half] = mean[r];
        if (rstd_out != nullptr) rstd_out[row + r * half] = rstd[r];
      }
    land(slot, single[0]);
    if (++slot == kRing) {
      slot = 0;
      phase ^= 1u;
    }
  }
}

template <int kPacked>
cudaError_t launch_stream_forward(const void* x, int bf16, int64_t ldx, const void* weight, const void* bias,
                                  int wbf16, int N, int D, float eps, void* y, int64_t ldy, float* mean,
                                  float* rstd, uint8_t* packed, int sms, cudaStream_t stream) {
  const int elt = bf16 ? 2 : 4;
  const RowLayout lay = row_layout(bf16, D, ldx, x, ldx, x, ldy, y, {weight, bias}, wbf16);
  if (sms < 8 || lay.narrow) return cudaErrorNotSupported;   // the caller has another kernel
  const int chunks = row_chunks(D, elt, !lay.whole), slot = 16 * chunks;
  const size_t params = static_cast<size_t>(slot / elt) * (wbf16 ? 2 : 4) *
                        ((weight != nullptr) + (bias != nullptr));
  const int grid = sms / 8 * 8;
  const StreamShape s = stream_shape(chunks, (static_cast<int64_t>(N) + 1) / 2, kForwardBlock,
                                     static_cast<size_t>(slot) * 2 * (kRing + (lay.apart ? 1 : 0)), params,
                                     grid);
  // Streaming pays from one row per group of a full CTA. bf16, streamed / one row per group of
  // a larger grid: D = 1024, N = 608 3.9 / 3.1 us, 1824 4.1 / 4.2, 4864 7.2 / 9.0; D = 4096,
  // N = 304 3.9 / 3.9, 912 6.5 / 8.8, 4864 17.8 / 25.0.
  if (s.groups == 0 || N < static_cast<int64_t>(kForwardBlock / s.R) * grid)
    return cudaErrorNotSupported;
  return with_stream_types(bf16, wbf16, !lay.whole, [&](auto b, auto wb, auto ragged) {
    return with_stream_vectors((chunks + s.R - 1) / s.R, [&](auto nv) {
      auto kern = norm_stream_kernel<b(), wb(), ragged(), nv(), kPacked>;
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(s.smem));
      if (e != cudaSuccess) return e;
      kern<<<grid, s.groups * s.R, s.smem, stream>>>(x, ldx, weight, bias, N, D, eps, y, ldy, mean,
                                                    rstd, packed, s.R, slot, lay.apart);
      return cudaGetLastError();
    });
  });
}

}  // namespace
}  // namespace flce
