// The ring through which the streaming layer-norm kernels read their rows.
//
// A CTA has groups of R threads, each of which walks its own rows through a ring of kRing
// turns' rows in shared memory, filled by the bulk-copy engine: one thread starts a row's
// copy, nobody spends registers or instructions on loads in flight, and 100 KB or more per SM
// are on their way at any time.
//
// The engine copies 16-byte chunks. Rows that begin or end inside a chunk (kRagged) keep
// their place relative to the chunks: whole chunks are copied, the few elements outside them
// go through a register of a thread that stores them a turn later, and a thread owns chunks,
// masking what lies beside the row. Where the rows read agree in their offsets from
// a 16-byte boundary, which repeat every 8 rows at most, a grid of a multiple of 8 CTAs that
// takes rows blockIdx.x, blockIdx.x + gridDim.x, ... has one offset per CTA, so that columns
// stay with their threads (for the sums over rows) and the weights are laid out once.
#pragma once

#include <cstdint>

#include "flce_norm.cuh"
#include "ptx.cuh"

namespace flce {
namespace {

constexpr int kStreamVectors = 4;    // 16-byte vectors of a row per thread at most
constexpr uint64_t kStreamWaitNs = 2000000000ull;

// Barrier of the R threads of a group.
__device__ __forceinline__ void group_sync(int group, int R) {
  if (R == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(R) : "memory");
}

// Sum over the group, the same in all of its threads; one barrier. `slots` (a float2 per warp
// of the CTA) must not be written again before another barrier of the group.
__device__ __forceinline__ float2 stream_sum2(float2 v, int group, int R, float2* slots) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (R == 32) return v;
  if (lane == 0) slots[warp] = v;
  group_sync(group, R);
  const int per = R >> 5, base = group * per;
  float2 s = slots[base];
#pragma unroll 4
  for (int w = 1; w < per; ++w) {
    const float2 o = slots[base + w];
    s.x += o.x;
    s.y += o.y;
  }
  return s;
}
// How the rows of a CTA lie in their 16-byte chunks of VW elements.
template <int kElt, bool kRagged>
struct RowPlace {
  static constexpr int VW = 16 / kElt;
  int s, tail, chunks;   // elements of the first chunk before the row, of the last one in it if not all
  __device__ RowPlace(const void* row, int D) {
    s = kRagged ? static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / kElt : 0;
    tail = kRagged ? (s + D) % VW : 0;
    chunks = kRagged ? (s + D + VW - 1) / VW : D / VW;
  }
  __device__ int head() const { return kRagged && s > 0 ? VW - s : 0; }
  __device__ uint32_t whole_bytes(int D) const { return static_cast<uint32_t>((D - head() - tail) * kElt); }
  // one thread: starts the copy of the row's whole chunks
  __device__ void copy(uint32_t slot, const uint8_t* row, int D, uint32_t bar) const {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            slot + (kRagged && s > 0 ? 16u : 0u)),
        "l"(row + head() * kElt), "r"(whole_bytes(D)), "r"(bar)
        : "memory");
  }
  // The q-th element (of 16) that is in no whole chunk, or -1: read by a thread of its own,
  // which writes it to the ring a turn later.
  __device__ int single(int q, int D) const {
    const int h = head();
    return q < h ? q : q < h + tail ? D - tail + q - h : -1;
  }
  __device__ uint32_t read_single(const uint8_t* row, int q, int D) const {
    const int i = single(q, D);
    if (i < 0) return 0;
    return kElt == 2 ? reinterpret_cast<const uint16_t*>(row)[i] : reinterpret_cast<const uint32_t*>(row)[i];
  }
  __device__ void write_single(uint8_t* slot, int q, int D, uint32_t bits) const {
    const int i = single(q, D);
    if (i < 0) return;
    if (kElt == 2) reinterpret_cast<uint16_t*>(slot)[s + i] = static_cast<uint16_t>(bits);
    else reinterpret_cast<uint32_t*>(slot)[s + i] = bits;
  }
  __device__ bool edge(int c) const { return kRagged && ((c == 0 && s > 0) || (c == chunks - 1 && tail > 0)); }
  __device__ bool in_row(int c, int e, int D) const {
    const int i = c * VW + e - s;
    return i >= 0 && i < D;
  }
  // zeros in place of what chunk c has beside the row
  __device__ void mask(float (&v)[VW], int c, int D) const {
    if (edge(c)) {
#pragma unroll
      for (int e = 0; e < VW; ++e) v[e] = in_row(c, e, D) ? v[e] : 0.f;
    }
  }
  // chunk c to the row at element row_at of p, which lies in its chunks in the same way
  template <int kBf16>
  __device__ void store(void* p, int64_t row_at, const float (&v)[VW], int c, int D) const {
    if (edge(c)) {
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (in_row(c, e, D)) store_from_f32(p, row_at + c * VW + e - s, v[e], kBf16);
    } else {
      Pack<kBf16, VW>::store(p, row_at + c * VW - s, v);
    }
  }
  // The group copies a row from `staged`, where it lies as the rows read do, to `row`, which
  // may lie in its chunks in another way: each whole chunk there is put together from two
  // here.
  __device__ void copy_out(const uint8_t* staged, uint8_t* row, int D, int t, int R) const {
    const int so = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / kElt;
    const int shift = ((s - so) & (VW - 1)) * kElt, q = shift >> 2, bits = (shift & 3) * 8;
    for (int i = t * VW - so; i < D; i += R * VW) {
      if (i >= 0 && i + VW <= D) {
        const uint4* const from = reinterpret_cast<const uint4*>(staged) + (i + s) / VW;
        uint4 o = from[0];
        if (shift != 0) {
          const uint4 n = from[1];
          const uint32_t w[8] = {o.x, o.y, o.z, o.w, n.x, n.y, n.z, n.w};
          uint32_t u[5];
#pragma unroll
          for (int k = 0; k < 5; ++k)
            u[k] = q == 0 ? w[k] : q == 1 ? w[k + 1] : q == 2 ? w[k + 2] : w[(k + 3) & 7];
          o = make_uint4(__funnelshift_r(u[0], u[1], bits), __funnelshift_r(u[1], u[2], bits),
                         __funnelshift_r(u[2], u[3], bits), __funnelshift_r(u[3], u[4], bits));
        }
        *reinterpret_cast<uint4*>(row + i * kElt) = o;
      } else {
        for (int e = i < 0 ? 0 : i; e < i + VW && e < D; ++e) {
          if (kElt == 2)
            reinterpret_cast<uint16_t*>(row)[e] = reinterpret_cast<const uint16_t*>(staged)[s + e];
          else
            reinterpret_cast<uint32_t*>(row)[e] = reinterpret_cast<const uint32_t*>(staged)[s + e];
        }
      }
    }
  }
};

// After a copy that did not come in time: waits, again with a limit, for those of a group's
// ring (turns `turn_row`, `turn_row` + step, ... from `slot` on), so that none is in flight
// when the memory is given back. No further one is started.
static __device__ __noinline__ void drain_ring(uint64_t* full, int ring, int slot, uint32_t phase,
                                        int64_t turn_row, int64_t step, int N) {
  const volatile int never = 0;
  for (int d = 0; d < ring && turn_row + d * step < N; ++d) {
    const int at = slot + d;
    mbar_wait_bounded(smem_u32(full + at % ring), phase ^ (at >= ring ? 1u : 0u), 1000000000ull, &never);
  }
}

// weight and bias (either may be null) to shared memory, in the places of the rows' chunks
// (zeros beside the row)
template <int kWbf16, int VW, bool kRagged>
__device__ __forceinline__ void stage_params(const void* w, uint8_t* to_w, const void* b, uint8_t* to_b,
                                             int s, int chunks, int D) {
  if constexpr (!kRagged) {
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
      Param<kWbf16, VW> p;
      if (w != nullptr) {
        p.load(w, c * VW, 0.f);
        p.save(to_w, c * VW);
      }
      if (b != nullptr) {
        p.load(b, c * VW, 0.f);
        p.save(to_b, c * VW);
      }
    }
  } else {
#pragma unroll 4
    for (int j = threadIdx.x; j < chunks * VW; j += blockDim.x) {
      const int i = j - s;
      const bool in = i >= 0 && i < D;
      if (w != nullptr) store_from_f32(to_w, j, in ? load_as_f32(w, i, kWbf16) : 0.f, kWbf16);
      if (b != nullptr) store_from_f32(to_b, j, in ? load_as_f32(b, i, kWbf16) : 0.f, kWbf16);
    }
  }
}

// Chunks that a row of D elements can touch, and its bytes in the ring.
inline int row_chunks(int D, int elt, bool ragged) {
  const int vw = 16 / elt;
  return ragged ? (D + 2 * vw - 2) / vw : D / vw;
}

// How rows lie in their chunks: `whole` ones, or alike in the rows that are read (two strides
// and two addresses), or neither (the kernels do not take them). `apart`: the output's differ,
// and are staged in shared memory on their way out; `narrow`: that, where rows are read
// 8 bytes at a time anyway, costs more than it gives: 8000 x 4096 bf16 in rows of 4100 62.6 us
// forward and 96.8 backward, by the kernels of rows in registers 40.9 and 57.9 (but 8000 x 4001
// in rows of 4004, 2 bytes at a time, 55.9 and 79.7, there 77.6 and 97.0).
struct RowLayout {
  bool whole, alike, apart, narrow;
};
inline RowLayout row_layout(int bf16, int D, int64_t ld, const void* p, int64_t ld2, const void* p2,
                            int64_t ldo, const void* o, std::initializer_list<const void*> params,
                            int wbf16) {
  const int elt = bf16 ? 2 : 4;
  auto differ = [&](int64_t s, const void* q) {
    return (s - ld) * elt % 16 != 0 ||
           (reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) % 16 != 0;
  };
  RowLayout r;
  r.whole = access_width(bf16, D, {ld, ld2, ldo}, {p, p2, o}, params, wbf16) == 16 / elt;
  r.alike = !differ(ld2, p2);
  r.apart = !r.whole && differ(ldo, o);
  r.narrow = r.apart && access_width(bf16, D, {ld, ld2}, {p, p2}, {}, 0) * elt >= 8;
  return r;
}

// Threads per row, a multiple of 32, and groups per CTA of at most `block` threads whose
// rings (`ring_bytes` each) fit beside `fixed` bytes; 0 groups if none does.
struct StreamShape {
  int R, groups;
  size_t smem;
};
inline StreamShape stream_shape(int nvec, int64_t turns, int block, size_t ring_bytes, size_t fixed,
                                int sms) {
  StreamShape s;
  s.R = ((nvec + kStreamVectors - 1) / kStreamVectors + 31) / 32 * 32;
  s.groups = block / s.R;
  constexpr size_t kMost = 224 * 1024;
  while (s.groups > 0 && fixed + s.groups * ring_bytes > kMost) --s.groups;
  const int64_t per_sm = (turns + sms - 1) / sms;   // few rows: spread over the SMs
  if (s.groups > per_sm) s.groups = static_cast<int>(per_sm);
  s.smem = fixed + static_cast<size_t>(s.groups) * ring_bytes;
  return s;
}

// f(vectors per thread): all but the last are inside the row for every thread.
template <typename F>
cudaError_t with_stream_vectors(int per, F&& f) {
  static_assert(kStreamVectors == 4, "the cases below");
  if (per <= 2) return f(std::integral_constant<int, 2>{});
  if (per == 3) return f(std::integral_constant<int, 3>{});
  return f(std::integral_constant<int, 4>{});
}

// f(bf16, wbf16, ragged) with the values as compile-time constants.
template <typename F>
cudaError_t with_stream_types(int bf16, int wbf16, bool ragged, F&& f) {
  using One = std::integral_constant<int, 1>;
  using Zero = std::integral_constant<int, 0>;
  auto types = [&](auto r) {
    if (bf16) return wbf16 ? f(One{}, One{}, r) : f(One{}, Zero{}, r);
    return wbf16 ? f(Zero{}, One{}, r) : f(Zero{}, Zero{}, r);
  };
  return ragged ? types(One{}) : types(Zero{});
}

}  // namespace
}  // namespace flce
