// Global 2-norm of many gradients, and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2), c = min(1, max_norm / (norm + 1e-6)),
//   out = c g
//
// The tensors are cut into pieces of kPieceBytes; the pieces of all tensors of a launch
// are dealt to the CTAs in turn. The table of tensors travels in the kernel's parameters
// (nothing is copied to the device, so a call can be captured), kTableTensors at a time.
// Squares are summed in fp32 within a piece and thread (32 at most) and joined in fp64 in
// a fixed order, one partial per CTA and launch. Each CTA of the scaling launch adds up
// the partials itself: the same sum in the same order, with no third launch between.
//
// Bound by HBM: a read for the norm, then a read and a write. 1.8 GB of bf16 gradients in 49
// tensors 828 us, 790 at the copy rate; 64 small fp32 tensors (1.5 MB) 10.3 us a call, of which
// the host spends 10.
#include <cmath>
#include <cstdint>

#include "flce_clip.h"
#include "flce_internal.h"
#include "flce_launch.cuh"

namespace flce {

namespace {

constexpr int kClipThreads = 512;
constexpr int kPieceBytes = 32 << 10;

// Sum over the CTA, valid in warp 0. The fp64 units add two lanes a cycle: warp 0 adds up
// 16 values per lane, then the lanes (500 cycles against the 1300 of shuffles in every warp).
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double block_sum(double v, double* s_all) {
  s_all[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  double r = s_all[threadIdx.x];
#pragma unroll
  for (int j = 1; j < kClipThreads / 32; ++j) r += s_all[threadIdx.x + 32 * j];
  return warp_sum(r);
}

// The tensor that holds piece `p`: the last whose first piece is at most p. Tensors of one
// size are found at once, others by halving.
__device__ __forceinline__ int tensor_of(const ClipTable& tab, int p) {
  const int guess = min(static_cast<int>(static_cast<float>(p) * tab.density), tab.count - 1);
  if (tab.first[guess] <= p && (guess + 1 == tab.count || tab.first[guess + 1] > p)) return guess;
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Sum of squares of n elements from p, this thread's share. The vectors lie between the
// first and the last 16-byte boundary; the elements outside are read singly.
__device__ __forceinline__ float squares(const uint8_t* p, int n, int bf16) {
  const int elt = bf16 ? 2 : 4, E = 16 / elt;
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / elt;
  int head = mis ? E - mis : 0;
  if (head > n) head = n;
  const int nvec = (n - head) / E, tail = head + nvec * E;
  float s0 = 0.f, s1 = 0.f;
  const uint4* vec = reinterpret_cast<const uint4*>(p + head * elt);
#pragma unroll 4
  for (int v = threadIdx.x; v < nvec; v += kClipThreads) {
    const uint4 q = __ldg(vec + v);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (bf16) {
        const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
        s0 = fmaf(a, a, s0);
        s1 = fmaf(b, b, s1);
      } else {
        const float a = __uint_as_float(w[i]);
        if (i & 1) s1 = fmaf(a, a, s1);
        else s0 = fmaf(a, a, s0);
      }
    }
  }
  const int singles = head + n - tail;
  if (static_cast<int>(threadIdx.x) < singles) {
    const int i = static_cast<int>(threadIdx.x) < head ? threadIdx.x : tail + threadIdx.x - head;
    const float a = bf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << 16)
                         : reinterpret_cast<const float*>(p)[i];
    s0 = fmaf(a, a, s0);
  }
  return s0 + s1;
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t w, float c) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
      : "=r"(r)
      : "f"(__uint_as_float(w & 0xFFFF0000u) * c), "f"(__uint_as_float(w << 16) * c));
  return r;
}

__device__ __forceinline__ void scale_piece(const uint8_t* p, uint8_t* q, int n, int bf16, float c) {
  const int elt = bf16 ? 2 : 4, E = 16 / elt;
  int head = n;
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) == 0) {
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / elt;
    head = mis ? E - mis : 0;
    if (head > n) head = n;
  }
  const int nvec = (n - head) / E, tail = head + nvec * E;
  const uint4* src = reinterpret_cast<const uint4*>(p + head * elt);
  uint4* dst = reinterpret_cast<uint4*>(q + head * elt);
#pragma unroll 4
  for (int v = threadIdx.x; v < nvec; v += kClipThreads) {
    uint4 w = src[v];
    if (bf16) {
      w = make_uint4(scale_pair(w.x, c), scale_pair(w.y, c), scale_pair(w.z, c), scale_pair(w.w, c));
    } else {
      w = make_uint4(__float_as_uint(__uint_as_float(w.x) * c), __float_as_uint(__uint_as_float(w.y) * c),
                     __float_as_uint(__uint_as_float(w.z) * c), __float_as_uint(__uint_as_float(w.w) * c));
    }
    dst[v] = w;
  }
  const int singles = head + n - tail;
  for (int j = threadIdx.x; j < singles; j += kClipThreads) {
    const int i = j < head ? j : tail + j - head;
    if (bf16)
      reinterpret_cast<uint16_t*>(q)[i] =
          static_cast<uint16_t>(scale_pair(reinterpret_cast<const uint16_t*>(p)[i], c) & 0xFFFFu);
    else
      reinterpret_cast<float*>(q)[i] = reinterpret_cast<const float*>(p)[i] * c;
  }
}

// Bytes and elements of piece `p` of a tensor.
struct Piece {
  int64_t at;   // first element
  int n;
};
__device__ __forceinline__ Piece piece_of(const ClipTable& tab, int t, int p) {
  const int per = kPieceBytes / (tab.bf16[t] ? 2 : 4);
  Piece r;
  r.at = static_cast<int64_t>(p - tab.first[t]) * per;
  const int64_t left = tab.numel[t] - r.at;
  r.n = left < per ? static_cast<int>(left) : per;
  return r;
}

__global__ void __launch_bounds__(kClipThreads, 4)
    grad_squares_kernel(const __grid_constant__ ClipTable tab, double* part) {
  __shared__ double s_all[kClipThreads];
  start_next_launch();
  double sum = 0.0;
  for (int p = blockIdx.x; p < tab.pieces; p += gridDim.x) {
    const int t = tensor_of(tab, p);
    const Piece c = piece_of(tab, t, p);
    const int elt = tab.bf16[t] ? 2 : 4;
    sum += static_cast<double>(squares(static_cast<const uint8_t*>(tab.src[t]) + c.at * elt, c.n, tab.bf16[t]));
  }
  const double total = block_sum(sum, s_all);
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kClipThreads, 4)
    grad_scale_kernel(const __grid_constant__ ClipTable tab, const double* part,
                      int parts, float max_norm, float* norm_out) {
  __shared__ float s_norm;
  wait_for_launch_before();   // the partials, and the last reads of what may be overwritten
  if (threadIdx.x < 32) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += 32) sum += part[i];
    s_norm = static_cast<float>(sqrt(warp_sum(sum)));
  }
  __syncthreads();
  const float norm = s_norm;
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float ratio = max_norm / (norm + 1e-6f);
  const float c = ratio > 1.f ? 1.f : ratio;   // NaN stays
  // backwards: the pieces that the norm read last are the ones still in L2
  for (int i = blockIdx.x; i < tab.pieces; i += gridDim.x) {
    const int p = tab.pieces - 1 - i;
    const int t = tensor_of(tab, p);
    if (tab.dst[t] == nullptr || (c == 1.f && tab.dst[t] == tab.src[t])) continue;
    const Piece q = piece_of(tab, t, p);
    const int64_t off = q.at * (tab.bf16[t] ? 2 : 4);
    scale_piece(static_cast<const uint8_t*>(tab.src[t]) + off, static_cast<uint8_t*>(tab.dst[t]) + off,
                q.n, tab.bf16[t], c);
  }
}

}  // namespace

int clip_piece_bytes() { return kPieceBytes; }

cudaError_t launch_grad_squares(const ClipTable& tab, double* part, int grid, cudaStream_t stream) {
  grad_squares_kernel<<<grid, kClipThreads, 0, stream>>>(tab, part);
  return cudaGetLastError();
}

cudaError_t launch_grad_scale(const ClipTable& tab, const double* part, int parts, float max_norm,
                              float* norm, int grid, cudaStream_t stream) {
  return launch_after(grad_scale_kernel, dim3(static_cast<unsigned>(grid)), dim3(kClipThreads), 0, stream,
                      tab, part, parts, max_norm, norm);
}

}  // namespace flce
