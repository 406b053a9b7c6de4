// The statistics of a softmax row that log probabilities and entropies are formed from,
// kept in the base-2 domain the hardware exponential works in.
//
// With c = log2(e) / temperature, a part of a row is
//   m = max z (raw logits), s = sum 2^d, t = sum 2^d d,  d_v = z_v c - r,
// with r = row_ref(m, c) a whole number next to m c: it is exact in fp32, so one FMA gives
// d with a single rounding of its own size, however far the logits are from 0, and parts
// join by factors 2^(r - r'). The token's own term is left out of s and t and added at the
// end, so that 1 - p of a confident token, and its log probability -log1p(others / its
// term), are no differences of nearly equal numbers.
#pragma once

#include <cmath>
#include <cstdint>

namespace flce {

constexpr float kLn2 = 0.6931471805599453f;
// A 2^d below 2^-200 is 0 in fp32 however d is rounded; the floor keeps d finite for
// logits of -inf, whose 2^d d would otherwise be 0 * -inf.
constexpr float kMinExponent = -200.f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Maximum that keeps a NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Logits whose m c leaves the range in which fp32 holds every whole number (a row of a type's
// lowest values, for one) have no such r: there d = (z - m) c.
constexpr float kMaxRef = 4194304.f;
__device__ __forceinline__ bool has_ref(float m, float c) { return fabsf(m * c) < kMaxRef; }
__device__ __forceinline__ float row_ref(float m, float c) { return rintf(m * c); }

// A log-sum-exp below this comes from a row whose every id is masked, with -inf or with
// the type's lowest value. Its gradient is 0: p = exp(x - lse) has no digits there.
constexpr float kMaskedLse = -1.0e30f;

struct RowPart {
  float m, s, t;
};

// d of a logit against the maximum m of its part.
__device__ __forceinline__ float row_exponent(float z, float m, float c) {
  return fmaxf(has_ref(m, c) ? fmaf(z, c, -row_ref(m, c)) : (z - m) * c, kMinExponent);
}

// What d of a part with maximum m becomes less by when the maximum becomes M >= m.
__device__ __forceinline__ float row_shift(float m, float M, float c) {
  float d;
  if (has_ref(m, c) && has_ref(M, c)) {
    d = row_ref(m, c) - row_ref(M, c);
  } else {   // r in place of m c on one side at most
    const float om = has_ref(m, c) ? fmaf(-m, c, row_ref(m, c)) : 0.f;
    const float oM = has_ref(M, c) ? fmaf(-M, c, row_ref(M, c)) : 0.f;
    d = (m - M) * c + (om - oM);
  }
  return fmaxf(d, kMinExponent);
}

// Joins b into a (either may be empty: m = -inf, s = t = 0). A NaN or +inf maximum
// stays one; s and t then have no meaning.
__device__ __forceinline__ void row_join(RowPart& a, const RowPart& b, float c) {
  const float M = max_nan(a.m, b.m);
  if (M == -INFINITY) return;
  const float da = row_shift(a.m, M, c), db = row_shift(b.m, M, c);
  const float fa = exp2_approx(da), fb = exp2_approx(db);
  a.t = fmaf(a.s, da, a.t) * fa + fmaf(b.s, db, b.t) * fb;
  a.s = a.s * fa + b.s * fb;
  a.m = M;
}

struct RowOut {
  float logprob, entropy, lse;
  float m, log_s;   // lse = m / temperature + log_s, for id_logprob
};

// Log probability of an id from its raw logit: no difference with lse, in which log_s
// drowns when the logits are far from 0. NaN in a row without a softmax.
__device__ __forceinline__ float id_logprob(const RowOut& r, float z, float inv_t) {
  return fmaf(z - r.m, inv_t, -r.log_s);
}

// The row's outputs from its joined part (the token's term left out), the raw logit zt
// of the token, and whether it has one. `inv_t` = 1 / temperature, c = log2(e) inv_t.
//
// Logarithms are of sums relative to the largest term e_m = 2^d_m, formed here as it was for the
// sums: where the others are 0 the logarithm and the entropy are 0, not the difference of two
// rounded numbers, log_s is never negative, and the largest id's log probability is the token's.
__device__ __forceinline__ RowOut row_finish(const RowPart& p, float zt, bool has_token,
                                             float inv_t, float c) {
  RowOut o;
  o.m = p.m;
  o.log_s = 0.f;
  if (!(p.m < INFINITY)) {   // NaN or +inf among the logits
    o.entropy = o.lse = o.log_s = __uint_as_float(0x7FC00000u);
    o.logprob = has_token ? o.lse : 0.f;
    return o;
  }
  if (p.m == -INFINITY) {    // every id is masked
    o.lse = -INFINITY;
    o.entropy = 0.f;
    o.logprob = has_token ? -INFINITY : 0.f;
    return o;
  }
  float dt = kMinExponent, et = 0.f;
  if (has_token) {
    dt = row_exponent(zt, p.m, c);
    et = exp2_approx(dt);
  }
  const float dm = row_exponent(p.m, p.m, c), em = exp2_approx(dm);
  // sums over the ids but the largest (the token, if it is that) of e and of e (d - d_m)
  const bool top = has_token && zt == p.m;
  const float s = top ? p.s : fmaxf(p.s + et - em, 0.f);
  const float t = top ? fmaf(-dm, p.s, p.t)
                      : fmaf(-dm, s, fmaf(et, dt, p.t) - __fmul_rn(em, dm));
  o.log_s = log1pf(s / em);
  o.lse = fmaf(p.m, inv_t, o.log_s);
  const float h = fmaf(-kLn2, t / (s + em), o.log_s);
  o.entropy = h < 0.f ? 0.f : h;
  // e_t < 2^-60: x_y - lse has no cancellation, and the quotient could overflow
  if (!has_token) o.logprob = 0.f;
  else if (top) o.logprob = -o.log_s;
  else o.logprob = et >= 0x1p-60f ? -log1pf(p.s / et) : id_logprob(o, zt, inv_t);
  return o;
}

// A row's gradient coefficients: dL/dz_v = p_v (A - B (log p_v + entropy)) off the
// token and `target` at it, everything divided by the temperature.
struct RowCoef {
  float lse, A, B, entropy, target;
};

__device__ __forceinline__ RowCoef row_coef(float lse, float entropy, float logprob, float a,
                                            float b, float c, bool has_token, float inv_t) {
  RowCoef r;
  if (!has_token) a = 0.f;
  r.lse = lse;
  r.entropy = b != 0.f ? entropy : 0.f;
  r.A = (c - a) * inv_t;
  r.B = b * inv_t;
  r.target = 0.f;
  if (lse != lse) r.A = lse;   // NaN in the row: NaN everywhere, also where p is 0
  if (lse < kMaskedLse) {   // every id is masked: no gradient
    r.lse = 3.0e38f;        // p = 0 for every finite logit
    r.A = r.B = r.entropy = 0.f;
    return r;
  }
  if (has_token) {
    const float lp = fmaxf(logprob, -1.0e4f);   // p log p of a masked token is 0
    const float p = expf(lp);
    r.target = (-expm1f(lp) * a + p * (c - b * (lp + r.entropy))) * inv_t;
    if (logprob != logprob) r.target = logprob;
  }
  return r;
}

// The token's own entry, given its logit: none at -inf. (The log probability does not tell: that
// of a token with the type's lowest value is -inf too, at temperatures below 1.)
__device__ __forceinline__ float target_entry(float target, float z) {
  return z == -INFINITY && target == target ? 0.f : target;
}

}  // namespace flce
