// Layer norm of many rows, backward: with h = (x - mean) rstd and g = dy weight,
//   dx = rstd (g - mean(g) - h mean(g h)), dweight = sum_rows dy h, dbias = sum_rows dy.
//
// x and dy come through the ring (flce_norm_stream.cuh). A thread owns the same columns, up to
// 32, of every row of its group: dweight and dbias add up in its registers while dx is
// formed from the same copy of the row, so x and dy are read once for all three. The
// groups' sums meet in shared memory at the end, one partial per CTA.
//
// One row of a turn, as the accumulators leave no registers for a second. 8192 x 4096 bf16 takes
// 40.8 us (4.9 TB/s) with the partials (their join 4, their writing 2), 16384 x 8192 148 us (5.5
// TB/s), 4000 x 4096 fp32 38.4 us (5.1 TB/s), 2000 x 8000 39.6 us; the rows' loads in registers
// instead of the ring 55, 175, 46, 50. Bound by latency: 23 instructions per element from 12 warps an
// SM, whose 168 registers a thread leave no room for more, keep half of the issue slots busy. Reading
// the slot again for dx, to hold less and run 16 warps, took 53 us.
// Ragged rows (loads in registers in brackets): 3001 x 1111 fp32 18.1 us (25.2), 16384 x 2730
// bf16 77 (109), 16000 x 4001 bf16 102 (179).
//
// kPacked: x comes as 8-bit records (flce_pack.cu) instead, 1.03 bytes a value, each copied whole.
// dy's place in its 16-byte chunks then is the thread's, and its codes are put together from the
// words they lie in; a chunk has one scale, or two where rows are ragged. 8192 x 4096 bf16 39.5 us (102 MB read
// instead of 134; 41.6 with one value an instruction), 16384 x 8192 145, 4000 x 4096 fp32 32.4 (from x 37.4),
// 3001 x 1111 fp32 16.0, 16000 x 4001 bf16 140 (from x 102: codes and scales of unaligned chunks).
#pragma once

#include <cstdint>

#include "flce_blocks.cuh"
#include "flce_launch.cuh"
#include "flce_norm_stream.cuh"
#include "flce_norm_stream.h"

namespace flce {

namespace {

// bf16: 64 accumulators and 64 values of the row, 168 registers a thread. fp32: half of both.
constexpr int kMostBlock = 512;
constexpr int backward_block(int bf16) { return bf16 ? 384 : kMostBlock; }
constexpr int kRing = 3;   // turns of a group in the ring, of one row of x and dy each

// A record's place in the ring: the bytes before it take the reads of a ragged row's first chunk.
constexpr int kRecordFront = 16;
inline int record_slot(int D) { return kRecordFront + static_cast<int>(packed_record(D)) + 16; }

// The codes of a chunk of VW elements from element o of a row on (o < 0 in a ragged row's first
// chunk), and the scales of its elements.
template <int VW, int kRagged>
struct ChunkCodes {
  uint32_t w[VW / 4], byte0, byte1;
  int split;   // elements before `split` have byte0's scale
  __device__ void load(const uint8_t* record, int codes, int o, bool ok) {
#pragma unroll
    for (int k = 0; k < VW / 4; ++k) w[k] = 0;
    byte0 = byte1 = 0;
    split = VW;
    if (!ok) return;
    if constexpr (!kRagged) {
#pragma unroll
      for (int k = 0; k < VW / 4; ++k) w[k] = reinterpret_cast<const uint32_t*>(record + o)[k];
      byte0 = record[codes + (o >> 5)];
    } else {
      const uint32_t* const from = reinterpret_cast<const uint32_t*>(record + (o & ~3));
#pragma unroll
      for (int k = 0; k < VW / 4; ++k) w[k] = __funnelshift_r(from[k], from[k + 1], (o & 3) * 8);
      const int b = o < 0 ? 0 : o >> 5;
      byte0 = record[codes + b];
      byte1 = record[codes + b + 1];
      split = 32 * (b + 1) - o;
    }
  }
  // the codes' values, without their scale
  __device__ void widen(float (&v)[VW]) const {
#pragma unroll
    for (int k = 0; k < VW / 4; ++k) {
      widen_e4m3x2(w[k], v[k * 4], v[k * 4 + 1]);
      widen_e4m3x2(w[k] >> 16, v[k * 4 + 2], v[k * 4 + 3]);
    }
  }
};

// x: rows of x, or (kPacked) records, ldx then in bytes.
template <int kBf16, int kWbf16, int kRagged, int kNv, int kPacked>
__global__ void __launch_bounds__(backward_block(kBf16), 1)
    norm_stream_grad_kernel(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                            const void* weight, const float* __restrict__ mean_in,
                            const float* __restrict__ rstd_in, int N, int D, void* dx,
                            int64_t lddx, float* part, void* dweight, void* dbias, int R,
                            int slot_bytes, int apart) {
  constexpr int kElt = kBf16 ? 2 : 4, VW = 16 / kElt;
  constexpr int kFetchers = kRagged ? 32 : 1;
  using E = Each<kPacked>;
  using P = Pack<kBf16, VW>;
  using Raw = typename P::Raw;
  using W = Param<kWbf16, VW>;
  extern __shared__ uint4 s_dyn[];
  __shared__ __align__(8) uint64_t s_full[kMostBlock / 32][kRing];
  __shared__ float2 s_sum[2][kMostBlock / 32];
  start_next_launch();   // the join's CTAs come as these go
  const int groups = static_cast<int>(blockDim.x) / R;
  const int group = threadIdx.x / R, t = threadIdx.x % R;
  const float inv_d = 1.f / static_cast<float>(D);
  const RowPlace<kElt, kRagged> place(
      kPacked ? static_cast<const uint8_t*>(dy) + blockIdx.x * lddy * kElt
              : static_cast<const uint8_t*>(x) + blockIdx.x * ldx * kElt,
      D);
  const int chunks = place.chunks;
  // [each group's ring, x and dy of each row, and a row on its way out][weight]
  const int codes = static_cast<int>(packed_codes(D));
  const int x_bytes = kPacked ? kRecordFront + static_cast<int>(packed_record(D)) + 16 : slot_bytes;
  // where turn `slot` has x, or (half = 1) dy; past the last, the row on its way out
  auto place_of = [&](int slot, int half) {
    return kPacked ? slot * (x_bytes + slot_bytes) + half * x_bytes : (slot * 2 + half) * slot_bytes;
  };
  const int extra = kRagged && apart ? 1 : 0;
  const int group_bytes = kPacked ? place_of(kRing, 0) + extra * slot_bytes : (kRing * 2 + extra) * slot_bytes;
  uint8_t* const ring = reinterpret_cast<uint8_t*>(s_dyn) + group * group_bytes;
  uint8_t* const staged = ring + place_of(kRing, 0);
  uint8_t* const s_w = reinterpret_cast<uint8_t*>(s_dyn) + groups * group_bytes;

  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = kRagged ? blockIdx.x + static_cast<int64_t>(gridDim.x) * group
                                : static_cast<int64_t>(blockIdx.x) * groups + group;
  // by the first 32 threads of a group, or its first
  auto fetch = [&](int64_t row, int slot, uint32_t& single) {
    if (row >= N) return;
    const uint8_t* const from_x = static_cast<const uint8_t*>(x) + row * ldx * (kPacked ? 1 : kElt);
    const uint8_t* const from_g = static_cast<const uint8_t*>(dy) + row * lddy * kElt;
    uint8_t* const to = ring + place_of(slot, 0);
    if (t == 0) {
      const uint32_t bar = smem_u32(&s_full[group][slot]);
      if constexpr (kPacked) {
        const uint32_t record = static_cast<uint32_t>(ldx);
        mbar_arrive_expect_tx(bar, record + place.whole_bytes(D));
        copy_bytes(smem_u32(to + kRecordFront), from_x, record, bar);
      } else {
        mbar_arrive_expect_tx(bar, 2 * place.whole_bytes(D));
        place.copy(smem_u32(to), from_x, D, bar);
      }
      place.copy(smem_u32(to + x_bytes), from_g, D, bar);
    }
    if (kRagged && (!kPacked || t >= 16))   // 16 lanes for x and for dy
      single = place.read_single(t < 16 ? from_x : from_g, t & 15, D);
  };
  auto land = [&](int slot, uint32_t single) {
    if (kRagged && t < 32 && (!kPacked || t >= 16))
      place.write_single(ring + place_of(slot, t >> 4), t & 15, D, single);
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
  stage_params<kWbf16, VW, kRagged>(weight, s_w, nullptr, nullptr, place.s, chunks, D);
#pragma unroll
  for (int k = 0; k < kRing; ++k) land(k, single[k]);
  __syncthreads();
  float dw[kNv][VW], db[kNv][VW];
#pragma unroll
  for (int k = 0; k < kNv; ++k)
#pragma unroll
    for (int e = 0; e < VW; ++e) dw[k][e] = db[k][e] = 0.f;
  float mean_next = first < N ? mean_in[first] : 0.f, rstd_next = first < N ? rstd_in[first] : 0.f;
  const volatile int never = 0;
  uint64_t limit = kStreamWaitNs;
  int slot = 0, turn = 0;
  uint32_t phase = 0;
  for (int64_t row = first; row < N; row += step, ++turn) {
    float mean = mean_next, rstd = rstd_next;
    if (row + step < N) {
      mean_next = mean_in[row + step];
      rstd_next = rstd_in[row + step];
    }
    // a copy that never came makes its row, and the sums, NaN
    if (!mbar_wait_bounded(smem_u32(&s_full[group][slot]), phase, limit, &never)) {
      rstd = __uint_as_float(0x7FC00000u);
      if (t == 0 && limit != 0) drain_ring(s_full[group], kRing, slot, phase, row, step, N);
      limit = 0;
    }
    const uint8_t* in_x = ring + place_of(slot, 0);
    const uint8_t* in_g = in_x + x_bytes;
    // elements past the row have dy = 0 and so count nowhere
    auto inside = [&](int k) { return k < kNv - 1 || t + k * R < chunks; };
    Raw rg[kNv];
    [[maybe_unused]] Raw rx[kNv];
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      if constexpr (!kPacked) rx[k] = P::load_if(in_x, (t + k * R) * VW, inside(k));
      rg[k] = P::load_if(in_g, (t + k * R) * VW, inside(k));
    }
    float g[kNv][VW], h[kNv][VW], s0[VW], s1[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) s0[e] = s1[e] = 0.f;
#pragma unroll
    for (int k = 0; k < kNv; ++k) {
      if constexpr (kPacked) {   // x~ is exact, so its difference from the mean is rounded once
        ChunkCodes<VW, kRagged> c;
        c.load(in_x + kRecordFront, codes, (t + k * R) * VW - place.s, inside(k));
        c.widen(h[k]);
        P::widen(rg[k], g[k]);
        const float scale0 = power_of_byte(c.byte0), scale1 = kRagged ? power_of_byte(c.byte1) : 0.f;
        const uint64_t less = pair(-mean, -mean), by = pair(rstd, rstd);
#pragma unroll
        for (int e = 0; e < VW; e += 2) {
          const uint64_t scale = pair(!kRagged || e < c.split ? scale0 : scale1,
                                      !kRagged || e + 1 < c.split ? scale0 : scale1);
          split(mul2(fma2(pair(h[k][e], h[k][e + 1]), scale, less), by), h[k][e], h[k][e + 1]);
        }
        place.mask(h[k], t + k * R, D);
        place.mask(g[k], t + k * R, D);
      } else {
        P::widen(rx[k], h[k]);
        P::widen(rg[k], g[k]);
        place.mask(h[k], t + k * R, D);
        place.mask(g[k], t + k * R, D);
#pragma unroll
        for (int e = 0; e < VW; ++e) h[k][e] = (h[k][e] - mean) * rstd;
      }
      E::fma(dw[k], g[k], h[k], dw[k]);
      E::add(db[k], g[k]);
      if (weight != nullptr) {
        W p;
        float w[VW];
        p.load_if(s_w, (t + k * R) * VW, inside(k));
        p.widen(w);
        E::mul(g[k], w);
      }
      E::add(s0, g[k]);
      E::fma(s1, g[k], h[k], s1);
    }
    const float2 sum =
        stream_sum2(make_float2(sum_n(s0), sum_n(s1)), group, R, s_sum[turn & 1]);
    if (R == 32) __syncwarp();
    if (t < kFetchers && limit != 0) {   // everyone has read the slot; those reads come before the copies' writes
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      fetch(row + kRing * step, slot, single[0]);
    }
    if (dx != nullptr) {
      const float mg = -rstd * sum.x * inv_d, mgh = -rstd * sum.y * inv_d;
#pragma unroll
      for (int k = 0; k < kNv; ++k) {
        if constexpr (kPacked) {
          const uint64_t by = pair(rstd, rstd), mgs = pair(mg, mg), mghs = pair(mgh, mgh);
#pragma unroll
          for (int e = 0; e < VW; e += 2)
            split(fma2(pair(g[k][e], g[k][e + 1]), by, fma2(pair(h[k][e], h[k][e + 1]), mghs, mgs)), g[k][e],
                  g[k][e + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < VW; ++e)
            g[k][e] = fmaf(g[k][e], rstd, fmaf(h[k][e], mgh, mg));
        }
        if (inside(k)) {
          if (kRagged && apart) P::store(staged, (t + k * R) * VW, g[k]);
          else place.template store<kBf16>(dx, row * lddx, g[k], t + k * R, D);
        }
      }
      if (kRagged && apart) {
        group_sync(group, R);
        place.copy_out(staged, static_cast<uint8_t*>(dx) + row * lddx * kElt, D, t, R);
      }
    }
    land(slot, single[0]);
    if (++slot == kRing) {
      slot = 0;
      phase ^= 1u;
    }
  }
  if (part == nullptr) return;
  // the groups' sums meet in place of the rings: [group][dweight, dbias][chunks]
  float* const cols = reinterpret_cast<float*>(s_dyn);
  const int width = slot_bytes / kElt;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kNv; ++k)
    if (t + k * R < chunks) {
      float* const p = cols + group * 2 * width + (t + k * R) * VW;
#pragma unroll
      for (int e = 0; e < VW; e += 4) {
        *reinterpret_cast<float4*>(p + e) =
            make_float4(dw[k][e], dw[k][e + 1], dw[k][e + 2], dw[k][e + 3]);
        *reinterpret_cast<float4*>(p + width + e) =
            make_float4(db[k][e], db[k][e + 1], db[k][e + 2], db[k][e + 3]);
      }
    }
  __syncthreads();
  if (!kRagged && gridDim.x > 1) {   // four columns at a time
#pragma unroll 4
    for (int i = 4 * threadIdx.x; i < 2 * D; i += 4 * blockDim.x) {
      float4 s = *reinterpret_cast<const float4*>(cols + i);
      for (int q = 1; q < groups; ++q) {
        const float4 o = *reinterpret_cast<const float4*>(cols + q * 2 * D + i);
        s = make_float4(s.x + o.x, s.y + o.y, s.z + o.z, s.w + o.w);
      }
      *reinterpret_cast<float4*>(part + static_cast<int64_t>(blockIdx.x) * 2 * D + i) = s;
    }
    return;
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
    const int j = place.s + (i < D ? i : i - D + width);
    float s = cols[j];
    for (int q = 1; q < groups; ++q) s += cols[q * 2 * width + j];
    if (gridDim.x > 1) {
      part[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = s;
    } else {
      void* const out = i < D ? dweight : dbias;
      if (out != nullptr) store_from_f32(out, i < D ? i : i - D, s, kWbf16);
    }
  }
}

template <int kPacked>
cudaError_t launch_stream_grad(const void* dy, int64_t lddy, const void* x, int bf16, int64_t ldx,
                               const void* weight, int wbf16, const float* mean, const float* rstd, int N,
                               int D, void* dx, int64_t lddx, void* dweight, void* dbias, float* part,
                               int* ranges, int sms, cudaStream_t stream) {
  const int elt = bf16 ? 2 : 4;
  // (without dx as with a dense one, so that dweight does not depend on that)
  const RowLayout lay = row_layout(bf16, D, kPacked ? lddy : ldx, kPacked ? dy : x, lddy, dy,
                                   dx != nullptr ? lddx : D, dx, {weight}, wbf16);
  if (!lay.alike || lay.narrow || sms < 8) return cudaErrorNotSupported;   // the caller has another kernel
  const int chunks = row_chunks(D, elt, !lay.whole), slot = 16 * chunks;
  const size_t params =
      weight != nullptr ? static_cast<size_t>(slot / elt) * (wbf16 ? 2 : 4) : 0;
  const int most = sms / 8 * 8;
  const size_t turn = slot + (kPacked ? record_slot(D) : slot);
  const StreamShape s =
      stream_shape(chunks, N, backward_block(bf16), kRing * turn + (lay.apart ? slot : 0), params, most);
  // Streaming pays from 1.5 MB, or for long rows. bf16, streamed / by the kernel of rows in
  // registers: D = 1024, N = 304 10.3 / 7.0 us, 912 9.0 / 10.5, 4864 15.9 / 17.2; D = 4096,
  // N = 64 9.5 / 9.3, 304 12.6 / 20.5, 4864 31.5 / 40.6; D = 8192, N = 1 10.3 / 12.6.
  const int64_t row = static_cast<int64_t>(D) * (bf16 ? 2 : 4);
  if (s.groups == 0 || (N * row < 1536 * 1024 && row < 16 * 1024)) return cudaErrorNotSupported;
  static_assert(kRing * (2 + (kPacked ? 1 : 2)) >= 2 * 4, "the groups' sums fit in place of their rings");
  const int64_t want = N <= most ? N : ((N + s.groups - 1) / s.groups + 7) / 8 * 8;
  const int grid = static_cast<int>(want < most ? want : most);
  *ranges = grid;
  return with_stream_types(bf16, wbf16, !lay.whole, [&](auto b, auto wb, auto ragged) {
    return with_stream_vectors((chunks + s.R - 1) / s.R, [&](auto nv) {
      auto kern = norm_stream_grad_kernel<b(), wb(), ragged(), nv(), kPacked>;
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(s.smem));
      if (e != cudaSuccess) return e;
      kern<<<grid, s.groups * s.R, s.smem, stream>>>(dy, lddy, x, ldx, weight, mean, rstd, N, D, dx,
                                                     lddx, part, dweight, dbias, s.R, slot, lay.apart);
      return cudaGetLastError();
    });
  });
}

}  // namespace
}  // namespace flce
