// C ABI of the operators around the head (declared in include/flce_ops.h): argument
// checks, workspace layout and launch sequences.
//
// Launch sequences:
//   flce_token_logprobs            one kernel
//   flce_token_logprobs_backward   one kernel
//   flce_linear_token_logprobs     up to 128 tokens: the padded copies of the tokens (up to 64),
//                                  their product, the kernel of flce_token_logprobs over its
//                                  logits; else the log-probability GEMM, then the join of its
//                                  vocabulary ranges
//   flce_linear_token_logprobs_backward   row coefficients, then per token block and
//                                  vocabulary chunk the gradient GEMM and the dH / dW
//                                  products (launch_backward_products)
//   flce_layer_norm                one kernel
//   flce_layer_norm_backward       dx with partial column sums, then their join; hidden sizes
//                                  beyond what a CTA holds: column sums, dx, the join
//   flce_clip_grads                per table of tensors the squares, then per table the scaling
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/flce_ops.h"
#include "flce_clip.h"
#include "flce_gemm_few.h"
#include "flce_host.h"

namespace flce {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t elem_size(int32_t dtype) { return dtype == FLCE_DTYPE_BF16 ? 2 : 4; }
bool known_dtype(int32_t dtype) { return dtype == FLCE_DTYPE_F32 || dtype == FLCE_DTYPE_BF16; }

int check_logprob_options(const flce_logprob_options& o, int64_t V) {
  if (o.top_k < 0 || o.top_k > FLCE_MAX_TOP_K || o.top_k > V) return FLCE_ERR_OPTION;
  if (!(o.temperature >= 1e-6f && o.temperature <= 1e6f)) return FLCE_ERR_OPTION;
  if (!known_dtype(o.dw_dtype) || o.timeout_ns < 0) return FLCE_ERR_OPTION;
  return FLCE_OK;
}

flce_logprob_options logprob_options(const flce_logprob_options* opt) {
  flce_logprob_options o;
  flce_default_logprob_options(&o);
  if (opt != nullptr) o = *opt;
  return o;
}

int check_rows(int64_t N, int64_t V) {
  return (N < 0 || V < 1 || N > (int64_t(1) << 30) || V > (int64_t(1) << 30)) ? FLCE_ERR_SHAPE
                                                                               : FLCE_OK;
}

// The GB300 has 76 SM pairs; the ranges of the forward pass are planned for them, so
// that the workspace does not depend on a device being there.
constexpr int kPlanPairs = 76;

// Up to this many tokens the forward pass takes the logits of all of them (the kernel for few
// tokens) and then their rows; above it the large GEMM, which does not store them. In us with 5
// alternatives, here / by the GEMM, for 1, 64 and 128 tokens: D = 4096, V = 128256 168 / 880,
// 177 / 209, 196 / 208; D = 2048, V = 128256 90 / 486, 100 / 123, 113 / 117; D = 1024, V = 32000
// 22 / 98, 24 / 49, 27 / 49; D = 512, V = 8000 11 / 37, 13 / 37, 13 / 33. Without alternatives the
// GEMM is level from 96 tokens on at the first (192 / 193 at 128) and ahead at the second (109 / 99).
constexpr int64_t kFewTokens = 128;

struct LogpPlan {
  Plan P;
  bool few = false;
  int64_t ldz = 0;
  size_t off_pad = 0, off_z = 0;
  size_t off_part = 0, off_zt = 0, off_lists = 0, off_bounds = 0, off_coef = 0, off_target = 0, total = 0;
};

int make_logp_plan(int64_t N, int64_t D, int64_t V, const flce_logprob_options& o, bool backward,
                   LogpPlan* out) {
  LogpPlan L;
  flce_options fo;
  flce_default_options(&fo);
  fo.dw_dtype = o.dw_dtype;
  fo.v_splits = 1;
  if (N == 0) {
    *out = L;
    return FLCE_OK;
  }
  if (!backward && N <= kFewTokens) {
    L.few = true;
    L.ldz = static_cast<int64_t>(align_up(static_cast<size_t>(V), 4));
    L.off_pad = 0;
    L.off_z = align_up(static_cast<size_t>(kFewPadRows) * D * 2, 256);
    L.total = L.off_z + static_cast<size_t>(N) * L.ldz * 4;
    *out = L;
    return FLCE_OK;
  }
  if (!backward)
    // a ranking's entries hold 16 bits of column
    fo.v_splits = std::max(choose_splits(static_cast<int>(ceil_div(N, BM * kCtaGroup)),
                                         static_cast<int>(ceil_div(V, BN)), kPlanPairs),
                           static_cast<int>(ceil_div(ceil_div(V, BN), kMaxRangeTiles)));
  const int rc = make_plan(N, D, V, fo, 2 * kPlanPairs, &L.P, backward);
  if (rc != FLCE_OK) return rc;
  size_t off = backward ? L.P.total : 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  if (backward) {
    L.off_coef = take(static_cast<size_t>(N) * 16);
    L.off_target = take(static_cast<size_t>(N) * 4);
  } else {
    const size_t slots = static_cast<size_t>(L.P.splits) * L.P.part_stride * BM;
    L.off_part = take(slots * 16);
    L.off_zt = take(static_cast<size_t>(N) * 4);
    L.off_lists = take(slots * static_cast<size_t>(o.top_k) * 8);
    L.off_bounds = take(o.top_k > 0 ? static_cast<size_t>(N) * 4 : 0);
  }
  L.total = off;
  *out = L;
  return FLCE_OK;
}

int few_token_logprobs(const LogpPlan& L, const uint16_t* H, const uint16_t* W,
                       const int32_t* tokens, int64_t N, int64_t D, int64_t V,
                       const flce_logprob_options& o, float* logprob, float* entropy, float* lse,
                       float* top_logprob, int32_t* top_id, uint8_t* ws, int32_t* status, int sms,
                       cudaStream_t st) {
  const int kn = few_tile(N);
  uint16_t* pad = reinterpret_cast<uint16_t*>(ws + L.off_pad);
  FewParams p{};
  p.N = static_cast<int>(N);
  p.V = static_cast<int>(V);
  p.k_blocks = static_cast<int>(ceil_div(D, BK));
  p.z = reinterpret_cast<float*>(ws + L.off_z);
  p.ldz = L.ldz;
  p.timeout_ns = o.timeout_ns > 0 ? o.timeout_ns : kDefaultTimeoutNs;
  p.status = status;
  // more than 64 tokens are read as they are (rows past N read as zero)
  const bool direct = kn == kFewPadRows;
  p.copies = kFewPadRows / kn;
  CUtensorMap mW, mW16, mH;
  if (!encode_bf16(&mW, W, D, V, D, BK, BM) || !encode_bf16(&mW16, W, D, V, D, BK, 16) ||
      !encode_bf16(&mH, direct ? H : pad, D, direct ? N : kFewPadRows, D, BK,
                   static_cast<uint32_t>(kn)))
    return FLCE_ERR_CUDA;
  if (!direct && launch_pad_tokens(H, p.N, static_cast<int>(D), kn, pad, st) != cudaSuccess)
    return FLCE_ERR_CUDA;
  if (launch_few_logits(kn, mW, mW16, mH, p, sms, st) != cudaSuccess) return FLCE_ERR_CUDA;
  return launch_logprob_rows(0, p.z, p.ldz * 4, tokens, p.N, p.V, o.ignore_index, o.top_k,
                             1.f / o.temperature, logprob, entropy, lse, top_logprob, top_id,
                             status, sms, p.timeout_ns, st) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

int linear_shape(int64_t N, int64_t D, int64_t V) {
  if (N < 0) return FLCE_ERR_SHAPE;
  return check_shape(N == 0 ? 1 : N, D, V);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

void flce_default_logprob_options(flce_logprob_options* opt) {
  if (opt == nullptr) return;
  std::memset(opt, 0, sizeof(*opt));
  opt->ignore_index = -100;
  opt->temperature = 1.0f;
  opt->dw_dtype = FLCE_DTYPE_F32;
}

int flce_token_logprobs(const void* logits, int32_t dtype, int64_t ld, const int32_t* tokens,
                        int64_t N, int64_t V, const flce_logprob_options* opt, float* logprob,
                        float* entropy, float* lse, float* top_logprob, int32_t* top_id,
                        int32_t* status, void* stream) {
  const flce_logprob_options o = logprob_options(opt);
  int rc = check_rows(N, V);
  if (rc != FLCE_OK) return rc;
  rc = check_logprob_options(o, V);
  if (rc != FLCE_OK) return rc;
  if (!known_dtype(dtype)) return FLCE_ERR_OPTION;
  if (ld < V) return FLCE_ERR_SHAPE;
  if (N == 0) return FLCE_OK;
  if (logits == nullptr || (o.top_k > 0 && (top_logprob == nullptr || top_id == nullptr)))
    return FLCE_ERR_NULL;
  if (!aligned(logits, elem_size(dtype)) || !aligned(tokens, 4) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_logprob, 4) ||
      !aligned(top_id, 4) || !aligned(status, 4))
    return FLCE_ERR_ALIGN;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  const int64_t elt = static_cast<int64_t>(elem_size(dtype));
  return launch_logprob_rows(dtype == FLCE_DTYPE_BF16, logits, ld * elt, tokens,
                             static_cast<int>(N), static_cast<int>(V), o.ignore_index, o.top_k,
                             1.f / o.temperature, logprob, entropy, lse, top_logprob, top_id,
                             status, sms, o.timeout_ns > 0 ? o.timeout_ns : kDefaultTimeoutNs,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

// The upstream gradients of a row and the forward results they need.
static int check_upstream(const float* logprob, const float* entropy, const float* lse,
                          const float* dlogprob, const float* dentropy, const float* dlse,
                          const int32_t* tokens) {
  if (dlogprob == nullptr && dentropy == nullptr && dlse == nullptr) return FLCE_ERR_NULL;
  if (lse == nullptr || (dentropy != nullptr && entropy == nullptr)) return FLCE_ERR_NULL;
  // a token's entry is formed from its log probability whatever gradient there is
  if (tokens != nullptr && logprob == nullptr) return FLCE_ERR_NULL;
  for (const void* p : {static_cast<const void*>(logprob), static_cast<const void*>(entropy),
                        static_cast<const void*>(lse), static_cast<const void*>(dlogprob),
                        static_cast<const void*>(dentropy), static_cast<const void*>(dlse),
                        static_cast<const void*>(tokens)})
    if (!aligned(p, 4)) return FLCE_ERR_ALIGN;
  return FLCE_OK;
}

int flce_token_logprobs_backward(const void* logits, int32_t dtype, int64_t ld,
                                 const int32_t* tokens, int64_t N, int64_t V,
                                 const flce_logprob_options* opt, const float* logprob,
                                 const float* entropy, const float* lse, const float* dlogprob,
                                 const float* dentropy, const float* dlse, void* dlogits,
                                 int64_t dld, void* stream) {
  flce_logprob_options o = logprob_options(opt);
  o.top_k = 0;
  int rc = check_rows(N, V);
  if (rc != FLCE_OK) return rc;
  rc = check_logprob_options(o, V);
  if (rc != FLCE_OK) return rc;
  if (!known_dtype(dtype)) return FLCE_ERR_OPTION;
  if (ld < V || dld < V) return FLCE_ERR_SHAPE;
  if (N == 0) return FLCE_OK;
  if (logits == nullptr || dlogits == nullptr) return FLCE_ERR_NULL;
  rc = check_upstream(logprob, entropy, lse, dlogprob, dentropy, dlse, tokens);
  if (rc != FLCE_OK) return rc;
  if (!aligned(logits, elem_size(dtype)) || !aligned(dlogits, elem_size(dtype)))
    return FLCE_ERR_ALIGN;
  if (logits == dlogits && ld != dld) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  const int64_t elt = static_cast<int64_t>(elem_size(dtype));
  return launch_logprob_grad(dtype == FLCE_DTYPE_BF16, logits, ld * elt, tokens,
                             static_cast<int>(N), static_cast<int>(V), o.ignore_index,
                             1.f / o.temperature, logprob, entropy, lse, dlogprob, dentropy, dlse,
                             dlogits, dld * elt, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

int flce_linear_logprobs_workspace_size(int64_t N, int64_t D, int64_t V,
                                        const flce_logprob_options* opt, int32_t backward,
                                        size_t* bytes) {
  if (bytes == nullptr) return FLCE_ERR_NULL;
  const flce_logprob_options o = logprob_options(opt);
  int rc = linear_shape(N, D, V);
  if (rc != FLCE_OK) return rc;
  rc = check_logprob_options(o, V);
  if (rc != FLCE_OK) return rc;
  LogpPlan L;
  rc = make_logp_plan(N, D, V, o, backward != 0, &L);
  if (rc != FLCE_OK) return rc;
  *bytes = L.total;
  return FLCE_OK;
}

int flce_linear_token_logprobs(const uint16_t* H, const uint16_t* W, const int32_t* tokens,
                               int64_t N, int64_t D, int64_t V, const flce_logprob_options* opt,
                               float* logprob, float* entropy, float* lse, float* top_logprob,
                               int32_t* top_id, void* workspace, size_t ws_bytes,
                               int32_t* status, void* stream) {
  const flce_logprob_options o = logprob_options(opt);
  int rc = linear_shape(N, D, V);
  if (rc != FLCE_OK) return rc;
  rc = check_logprob_options(o, V);
  if (rc != FLCE_OK) return rc;
  if (N == 0) return FLCE_OK;
  if (H == nullptr || W == nullptr || workspace == nullptr ||
      (o.top_k > 0 && (top_logprob == nullptr || top_id == nullptr)))
    return FLCE_ERR_NULL;
  if (!aligned(H, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(tokens, 4) ||
      !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse, 4) ||
      !aligned(top_logprob, 4) || !aligned(top_id, 4) || !aligned(status, 4))
    return FLCE_ERR_ALIGN;
  LogpPlan L;
  rc = make_logp_plan(N, D, V, o, false, &L);
  if (rc != FLCE_OK) return rc;
  if (ws_bytes < L.total) return FLCE_ERR_WORKSPACE;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (L.few)
    return few_token_logprobs(L, H, W, tokens, N, D, V, o, logprob, entropy, lse, top_logprob,
                              top_id, ws, status, sms, st);
  const Plan& P = L.P;
  const int cta = P.cta;
  CUtensorMap mH, mW;
  if (!encode_bf16(&mH, H, D, N, D, BK, BM) ||
      !encode_bf16(&mW, W, D, V, D, BK, static_cast<uint32_t>(BN / cta)))
    return FLCE_ERR_CUDA;
  GemmParams g{};
  g.m_blocks = P.m_blocks;
  g.n_blocks = P.v_tiles;
  g.k_blocks = static_cast<int>(ceil_div(D, BK));
  g.splits = P.splits;
  g.part_stride = P.part_stride;
  g.num_units = P.splits * P.m_blocks;
  g.group_m = std::min(P.m_blocks, 16);
  g.idesc = make_idesc_bf16_f32(P.tile_m, BN, 0, 0);
  g.timeout_ns = o.timeout_ns > 0 ? o.timeout_ns : kDefaultTimeoutNs;
  g.status = status;
  g.m_valid = static_cast<int>(N);
  g.n_valid = static_cast<int>(V);
  g.labels = tokens;
  g.ignore_index = o.ignore_index;
  g.inv_t = 1.f / o.temperature;
  g.exp_scale = kLog2e * g.inv_t;
  g.top_k = o.top_k;
  g.part4 = reinterpret_cast<float4*>(ws + L.off_part);
  g.zt = reinterpret_cast<float*>(ws + L.off_zt);
  g.lists = reinterpret_cast<uint64_t*>(ws + L.off_lists);
  g.bounds = reinterpret_cast<uint32_t*>(ws + L.off_bounds);
  if (o.top_k > 0 &&
      cudaMemsetAsync(g.bounds, 0, static_cast<size_t>(N) * 4, st) != cudaSuccess)
    return FLCE_ERR_CUDA;
  const int pairs = std::max(1, sms / cta);
  if (launch_gemm_logp(mH, mW, g, cta * std::min(g.num_units, pairs), st) != cudaSuccess)
    return FLCE_ERR_CUDA;
  return launch_logprob_merge(g.part4, g.zt, g.lists, tokens, g.m_valid, g.n_valid, P.part_stride,
                              P.splits, o.ignore_index, o.top_k, g.inv_t, logprob, entropy, lse,
                              top_logprob, top_id, status, st) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

int flce_linear_token_logprobs_backward(const uint16_t* H, const uint16_t* W,
                                        const int32_t* tokens, int64_t N, int64_t D, int64_t V,
                                        const flce_logprob_options* opt, const float* logprob,
                                        const float* entropy, const float* lse,
                                        const float* dlogprob, const float* dentropy,
                                        const float* dlse, uint16_t* dH, void* dW,
                                        void* workspace, size_t ws_bytes, int32_t* status,
                                        void* stream) {
  flce_logprob_options o = logprob_options(opt);
  o.top_k = 0;
  int rc = linear_shape(N, D, V);
  if (rc != FLCE_OK) return rc;
  rc = check_logprob_options(o, V);
  if (rc != FLCE_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    if (dW == nullptr) return FLCE_OK;
    const size_t bytes = static_cast<size_t>(V) * D * elem_size(o.dw_dtype);
    return cudaMemsetAsync(dW, 0, bytes, st) == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
  }
  if (H == nullptr || W == nullptr || workspace == nullptr || (dH == nullptr && dW == nullptr))
    return FLCE_ERR_NULL;
  rc = check_upstream(logprob, entropy, lse, dlogprob, dentropy, dlse, tokens);
  if (rc != FLCE_OK) return rc;
  if (!aligned(H, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(dH, 16) ||
      !aligned(dW, 16) || !aligned(status, 4))
    return FLCE_ERR_ALIGN;
  LogpPlan L;
  rc = make_logp_plan(N, D, V, o, true, &L);
  if (rc != FLCE_OK) return rc;
  if (ws_bytes < L.total) return FLCE_ERR_WORKSPACE;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  const Plan& P = L.P;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  CUtensorMap mH, mW;
  if (!encode_bf16(&mH, H, D, N, D, BK, BM) ||
      !encode_bf16(&mW, W, D, V, D, BK, static_cast<uint32_t>(BN / P.cta)))
    return FLCE_ERR_CUDA;
  BackwardProducts bp{};
  bp.H = H;
  bp.W = W;
  bp.h_k = &mH;
  bp.w_k = &mW;
  bp.launch_grad = launch_gemm_logp_grad;
  bp.grad.k_blocks = static_cast<int>(ceil_div(D, BK));
  bp.grad.idesc = make_idesc_bf16_f32(P.tile_m, BN, 0, 0);
  bp.grad.labels = tokens;
  bp.grad.ignore_index = o.ignore_index;
  bp.grad.inv_t = 1.f / o.temperature;
  float4* coef = reinterpret_cast<float4*>(ws + L.off_coef);
  float* target = reinterpret_cast<float*>(ws + L.off_target);
  bp.grad.coef = coef;
  bp.grad.target = target;
  bp.dH = dH;
  bp.dW = dW;
  bp.dw_bf16 = o.dw_dtype == FLCE_DTYPE_BF16;
  bp.G = reinterpret_cast<uint16_t*>(ws + P.off_g);
  bp.dh_acc = reinterpret_cast<float*>(ws + P.off_dhacc);
  bp.dw_acc = reinterpret_cast<float*>(ws + P.off_dwacc);
  bp.timeout_ns = o.timeout_ns > 0 ? o.timeout_ns : kDefaultTimeoutNs;
  bp.status = status;
  bp.sms = sms;
  bp.stream = st;
  if (launch_logprob_coef(tokens, static_cast<int>(N), static_cast<int>(V), o.ignore_index,
                          bp.grad.inv_t, logprob, entropy, lse, dlogprob, dentropy, dlse, coef,
                          target, st) != cudaSuccess)
    return FLCE_ERR_CUDA;
  KernelTrace none;
  return launch_backward_products(P, bp, none);
}

static int check_norm(int64_t N, int64_t D, int32_t dtype, int32_t wdtype) {
  if (N < 0 || N > (int64_t(1) << 30) || D < 1 || D > (int64_t(1) << 24)) return FLCE_ERR_SHAPE;
  return known_dtype(dtype) && known_dtype(wdtype) ? FLCE_OK : FLCE_ERR_OPTION;
}

int flce_layer_norm(const void* x, int32_t dtype, int64_t ldx, const void* weight,
                    const void* bias, int32_t wdtype, int64_t N, int64_t D, float eps, void* y,
                    int64_t ldy, float* mean, float* rstd, void* stream) {
  int rc = check_norm(N, D, dtype, wdtype);
  if (rc != FLCE_OK) return rc;
  if (!(eps >= 0.f) || std::isinf(eps)) return FLCE_ERR_OPTION;
  if (ldx < D || ldy < D) return FLCE_ERR_SHAPE;
  if (N == 0) return FLCE_OK;
  if (x == nullptr || y == nullptr) return FLCE_ERR_NULL;
  const size_t e = elem_size(dtype), ew = elem_size(wdtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(weight, ew) || !aligned(bias, ew) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return FLCE_ERR_ALIGN;
  if (x == y && ldx != ldy) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return launch_layer_norm(x, dtype == FLCE_DTYPE_BF16, ldx, weight, bias,
                           wdtype == FLCE_DTYPE_BF16, static_cast<int>(N), static_cast<int>(D),
                           eps, y, ldy, mean, rstd, sms,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

int flce_layer_norm_workspace_size(int64_t N, int64_t D, size_t* bytes) {
  if (bytes == nullptr) return FLCE_ERR_NULL;
  const int rc = check_norm(N, D, FLCE_DTYPE_F32, FLCE_DTYPE_F32);
  if (rc != FLCE_OK) return rc;
  *bytes = static_cast<size_t>(std::min<int64_t>(N, kNormRanges)) * 2 * static_cast<size_t>(D) * 4;
  return FLCE_OK;
}

int flce_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int32_t dtype,
                             int64_t ldx, const void* weight, int32_t wdtype, const float* mean,
                             const float* rstd, int64_t N, int64_t D, void* dx, int64_t lddx,
                             void* dweight, void* dbias, void* workspace, size_t ws_bytes,
                             void* stream) {
  int rc = check_norm(N, D, dtype, wdtype);
  if (rc != FLCE_OK) return rc;
  if (ldx < D || lddy < D || (dx != nullptr && lddx < D)) return FLCE_ERR_SHAPE;
  const bool columns = dweight != nullptr || dbias != nullptr;
  if (N > 0) {
    if (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr ||
        (columns && workspace == nullptr))
      return FLCE_ERR_NULL;
    const size_t e = elem_size(dtype), ew = elem_size(wdtype);
    if (!aligned(dy, e) || !aligned(x, e) || !aligned(dx, e) || !aligned(weight, ew) ||
        !aligned(dweight, ew) || !aligned(dbias, ew) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !aligned(workspace, 16))
      return FLCE_ERR_ALIGN;
    if ((dx == dy && lddx != lddy) || dx == x) return FLCE_ERR_OPTION;
    size_t need = 0;
    rc = flce_layer_norm_workspace_size(N, D, &need);
    if (rc != FLCE_OK) return rc;
    if (columns && ws_bytes < need) return FLCE_ERR_WORKSPACE;
  }
  if (N == 0 && !columns) return FLCE_OK;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return launch_layer_norm_backward(dy, lddy, x, dtype == FLCE_DTYPE_BF16, ldx, weight,
                                    wdtype == FLCE_DTYPE_BF16, mean, rstd, static_cast<int>(N),
                                    static_cast<int>(D), dx, lddx, dweight, dbias,
                                    static_cast<float*>(workspace), sms,
                                    static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

// One fp64 partial per CTA and table of tensors.
static constexpr int kClipMaxGrid = 1024;

int flce_clip_grads_workspace_size(int64_t count, size_t* bytes) {
  if (bytes == nullptr) return FLCE_ERR_NULL;
  if (count < 0 || count > (int64_t(1) << 24)) return FLCE_ERR_SHAPE;
  *bytes = static_cast<size_t>(std::max<int64_t>(1, ceil_div(count, kTableTensors))) *
           kClipMaxGrid * sizeof(double);
  return FLCE_OK;
}

int flce_clip_grads(const void* const* grads, void* const* outs, const int64_t* numel,
                    const int32_t* dtypes, int64_t count, float max_norm, float* norm,
                    void* workspace, size_t ws_bytes, void* stream) {
  size_t need = 0;
  int rc = flce_clip_grads_workspace_size(count, &need);
  if (rc != FLCE_OK) return rc;
  if (norm == nullptr || workspace == nullptr ||
      (count > 0 && (grads == nullptr || numel == nullptr || dtypes == nullptr)))
    return FLCE_ERR_NULL;
  if (!(max_norm >= 0.f)) return FLCE_ERR_OPTION;
  if (!aligned(norm, 4) || !aligned(workspace, 16)) return FLCE_ERR_ALIGN;
  if (ws_bytes < need) return FLCE_ERR_WORKSPACE;
  for (int64_t i = 0; i < count; ++i) {
    if (!known_dtype(dtypes[i])) return FLCE_ERR_OPTION;
    if (numel[i] < 0 || numel[i] > (int64_t(1) << 40)) return FLCE_ERR_SHAPE;
    if (numel[i] == 0) continue;
    if (grads[i] == nullptr || (outs != nullptr && outs[i] == nullptr)) return FLCE_ERR_NULL;
    if (!aligned(grads[i], elem_size(dtypes[i])) ||
        (outs != nullptr && !aligned(outs[i], elem_size(dtypes[i]))))
      return FLCE_ERR_ALIGN;
  }
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  const int max_grid = std::min(kClipMaxGrid, sms * 4);
  const int64_t piece = clip_piece_bytes();

  // Fills a table with tensors from `*at` on; false when none is left.
  auto next_table = [&](int64_t* at, ClipTable* t) -> bool {
    t->count = 0;
    int64_t pieces = 0;
    for (; *at < count && t->count < kTableTensors; ++*at) {
      const int64_t i = *at;
      if (numel[i] == 0) continue;
      const int64_t n = ceil_div(numel[i] * static_cast<int64_t>(elem_size(dtypes[i])), piece);
      if (pieces + n > INT32_MAX) {
        if (t->count > 0) break;
        return false;   // not reached: one tensor of 2^40 elements is 2^27 pieces
      }
      const int k = t->count++;
      t->src[k] = grads[i];
      t->dst[k] = outs != nullptr ? outs[i] : nullptr;
      t->numel[k] = numel[i];
      t->first[k] = static_cast<int>(pieces);
      t->bf16[k] = dtypes[i] == FLCE_DTYPE_BF16;
      pieces += n;
    }
    t->pieces = static_cast<int>(pieces);
    t->density = static_cast<float>(t->count) / static_cast<float>(std::max<int64_t>(pieces, 1));
    return t->count > 0;
  };

  int parts = 0;
  ClipTable tab;
  int64_t at = 0;
  int tables = 0;
  while (next_table(&at, &tab)) {
    const int grid = std::min(tab.pieces, max_grid);
    if (launch_grad_squares(tab, part + parts, grid, st) != cudaSuccess) return FLCE_ERR_CUDA;
    parts += grid;
    ++tables;
  }
  if (outs == nullptr || tables == 0) {   // the norm alone
    std::memset(&tab, 0, sizeof(tab));
    return launch_grad_scale(tab, part, parts, max_norm, norm, 1, st) == cudaSuccess
               ? FLCE_OK
               : FLCE_ERR_CUDA;
  }
  at = 0;
  for (int k = 0; next_table(&at, &tab); ++k)
    if (launch_grad_scale(tab, part, parts, max_norm, k == 0 ? norm : nullptr,
                          std::min(tab.pieces, max_grid), st) != cudaSuccess)
      return FLCE_ERR_CUDA;
  return FLCE_OK;
}

}  // extern "C"
