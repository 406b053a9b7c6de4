// Shared by the layer-norm kernels: accesses of 2 to 16 bytes, paired fp32 arithmetic.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include <initializer_list>
#include <type_traits>

namespace flce {
namespace {

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16)
              : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_from_f32(void* p, int64_t i, float v, int bf16) {
  if (bf16) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(v));
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(r & 0xFFFFu);
  } else {
    static_cast<float*>(p)[i] = v;
  }
}

template <int kBytes>
struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

// VW consecutive elements, loaded and stored as one access.
template <int kBf16, int VW>
struct Pack {
  static constexpr int kBytes = VW * (kBf16 ? 2 : 4);
  using Raw = typename RawOf<kBytes>::type;
  __device__ static Raw load(const void* p, int64_t i) {
    return *reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(p) + i * (kBf16 ? 2 : 4));
  }
  // zeros where not `ok`
  __device__ static Raw load_if(const void* p, int64_t i, bool ok) {
    Raw r{};
    if (ok) r = load(p, i);
    return r;
  }
  __device__ static void widen(Raw raw, float (&x)[VW]) {
    if constexpr (!kBf16) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
      for (int e = 0; e < VW; ++e) x[e] = __uint_as_float(w[e]);
    } else if constexpr (VW == 1) {
      x[0] = __uint_as_float(static_cast<uint32_t>(raw) << 16);
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
      for (int e = 0; e < VW; e += 2) {
        x[e] = __uint_as_float(w[e / 2] << 16);
        x[e + 1] = __uint_as_float(w[e / 2] & 0xFFFF0000u);
      }
    }
  }
  __device__ static Raw narrow(const float (&x)[VW]) {
    Raw raw;
    if constexpr (!kBf16) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
      for (int e = 0; e < VW; ++e) w[e] = __float_as_uint(x[e]);
    } else if constexpr (VW == 1) {
      uint32_t r;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(x[0]));
      raw = static_cast<uint16_t>(r & 0xFFFFu);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
      for (int e = 0; e < VW; e += 2)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e / 2]) : "f"(x[e + 1]), "f"(x[e]));
    }
    return raw;
  }
  __device__ static void store(void* p, int64_t i, const float (&x)[VW]) {
    *reinterpret_cast<Raw*>(static_cast<uint8_t*>(p) + i * (kBf16 ? 2 : 4)) = narrow(x);
  }
};

// VW values of weight or bias from element i, or `none` without one.
template <int VW>
__device__ __forceinline__ void load_param(const void* p, int i, int wbf16, float none,
                                           float (&v)[VW]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < VW; ++e) v[e] = none;
  } else if (wbf16) {
    Pack<1, VW>::widen(Pack<1, VW>::load(p, i), v);
  } else {
    constexpr int W4 = VW < 4 ? VW : 4;
#pragma unroll
    for (int k = 0; k < VW; k += W4) {
      float q[W4];
      Pack<0, W4>::widen(Pack<0, W4>::load(p, i + k), q);
#pragma unroll
      for (int e = 0; e < W4; ++e) v[k + e] = q[e];
    }
  }
}

// VW values of weight or bias, kept as loaded (16 bytes at a time at most).
template <int kWbf16, int VW>
struct Param {
  static constexpr int kStep = VW * (kWbf16 ? 2 : 4) > 16 ? 16 / (kWbf16 ? 2 : 4) : VW;
  using P = Pack<kWbf16, kStep>;
  typename P::Raw raw[VW / kStep];
  // from element i, or VW times `none` without a vector
  __device__ void load(const void* p, int i, float none) {
    if (p != nullptr) {
#pragma unroll
      for (int k = 0; k < VW / kStep; ++k) raw[k] = P::load(p, i + k * kStep);
    } else {
      float v[kStep];
#pragma unroll
      for (int e = 0; e < kStep; ++e) v[e] = none;
#pragma unroll
      for (int k = 0; k < VW / kStep; ++k) raw[k] = P::narrow(v);
    }
  }
  // zeros where not `ok`
  __device__ void load_if(const void* p, int i, bool ok) {
#pragma unroll
    for (int k = 0; k < VW / kStep; ++k) raw[k] = P::load_if(p, i + k * kStep, ok);
  }
  // as they are, to shared memory
  __device__ void save(uint8_t* p, int i) const {
#pragma unroll
    for (int k = 0; k < VW / kStep; ++k)
      *reinterpret_cast<typename P::Raw*>(p + (i + k * kStep) * (kWbf16 ? 2 : 4)) = raw[k];
  }
  __device__ void narrow(const float (&v)[VW]) {
#pragma unroll
    for (int k = 0; k < VW / kStep; ++k) {
      float q[kStep];
#pragma unroll
      for (int e = 0; e < kStep; ++e) q[e] = v[k * kStep + e];
      raw[k] = P::narrow(q);
    }
  }
  __device__ void widen(float (&v)[VW]) const {
#pragma unroll
    for (int k = 0; k < VW / kStep; ++k) {
      float q[kStep];
      P::widen(raw[k], q);
#pragma unroll
      for (int e = 0; e < kStep; ++e) v[k * kStep + e] = q[e];
    }
  }
};

// Pack-wide arithmetic.
template <int VW>
__device__ __forceinline__ void fma_n(float (&d)[VW], const float (&a)[VW], const float (&b)[VW],
                                      const float (&c)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; ++e) d[e] = fmaf(a[e], b[e], c[e]);
}
template <int VW>
__device__ __forceinline__ void add_n(float (&d)[VW], const float (&a)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; ++e) d[e] += a[e];
}
template <int VW>
__device__ __forceinline__ void mul_n(float (&d)[VW], const float (&a)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; ++e) d[e] *= a[e];
}
// Two values at a time, each rounded as by itself.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The above and more of them, kPairs: two values an instruction.
template <int kPairs>
struct Each {
  template <int VW>
  __device__ static void fma(float (&d)[VW], const float (&a)[VW], const float (&b)[VW], const float (&c)[VW]) {
    if constexpr (kPairs && VW % 2 == 0) {
#pragma unroll
      for (int e = 0; e < VW; e += 2)
        split(fma2(pair(a[e], a[e + 1]), pair(b[e], b[e + 1]), pair(c[e], c[e + 1])), d[e], d[e + 1]);
    } else {
      fma_n(d, a, b, c);
    }
  }
  template <int VW>
  __device__ static void add(float (&d)[VW], const float (&a)[VW]) {
    if constexpr (kPairs && VW % 2 == 0) {
#pragma unroll
      for (int e = 0; e < VW; e += 2) split(add2(pair(d[e], d[e + 1]), pair(a[e], a[e + 1])), d[e], d[e + 1]);
    } else {
      add_n(d, a);
    }
  }
  template <int VW>
  __device__ static void mul(float (&d)[VW], const float (&a)[VW]) {
    if constexpr (kPairs && VW % 2 == 0) {
#pragma unroll
      for (int e = 0; e < VW; e += 2) split(mul2(pair(d[e], d[e + 1]), pair(a[e], a[e + 1])), d[e], d[e + 1]);
    } else {
      mul_n(d, a);
    }
  }
};

template <int VW>
__device__ __forceinline__ float sum_n(const float (&a)[VW]) {
  float s = a[0];
#pragma unroll
  for (int e = 1; e < VW; ++e) s += a[e];
  return s;
}

// Threads of a row of nvec vectors, a power of two from `least` to `limit`: enough for `each` vectors
// apiece, and more while the rows alone do not fill a quarter of the GPU's threads.
inline int threads_of_row(int64_t rows, int nvec, int each, int least, int limit) {
  constexpr int64_t kQuarter = 152 * 512;
  int X = least;
  while (X < limit && X * each < nvec) X *= 2;
  while (X < limit && X < nvec && rows * X < kQuarter) X *= 2;
  return X;
}

// The widest access (elements) that D, the row strides and the addresses allow.
inline int access_width(int bf16, int D, std::initializer_list<int64_t> strides,
                 std::initializer_list<const void*> rows, std::initializer_list<const void*> params,
                 int wbf16) {
  const int elt = bf16 ? 2 : 4, welt = wbf16 ? 2 : 4;
  int vw = 16 / elt;
  auto fits = [&](int v) {
    if (D % v != 0) return false;
    for (int64_t s : strides)
      if (s % v != 0) return false;
    for (const void* p : rows)
      if (reinterpret_cast<uintptr_t>(p) % static_cast<unsigned>(v * elt) != 0) return false;
    for (const void* p : params) {
      const unsigned a = static_cast<unsigned>(v * welt < 16 ? v * welt : 16);
      if (reinterpret_cast<uintptr_t>(p) % a != 0) return false;
    }
    return true;
  };
  while (vw > 1 && !fits(vw)) vw /= 2;
  return vw;
}


}  // namespace
}  // namespace flce
