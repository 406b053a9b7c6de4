// C ABI of the embedding (declared in include/flce_embed.h): argument checks, workspace layout and
// launch sequences.
//
//   flce_embedding            one kernel
//   flce_embedding_backward   the sort of the tokens (one kernel up to 16384 of them, else three a
//                             radix pass), the ranges' sums with the zeros of the other rows, the join of the
//                             ids that cross ranges
#include <cmath>
#include <cstdint>

#include "../../include/flce_embed.h"
#include "flce_embed.h"
#include "flce_host.h"

namespace flce {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t elem_size(int32_t dtype) { return dtype == FLCE_DTYPE_BF16 ? 2 : 4; }
bool known_dtype(int32_t dtype) { return dtype == FLCE_DTYPE_F32 || dtype == FLCE_DTYPE_BF16; }

int check_embed_shape(int64_t N, int64_t V, int64_t D) {
  return N < 0 || N > (int64_t(1) << 30) || V < 1 || V > (int64_t(1) << 30) || D < 1 ||
                 D > (int64_t(1) << 24)
             ? FLCE_ERR_SHAPE
             : FLCE_OK;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_embedding(const void* weight, int32_t wdtype, int64_t ldw, const int32_t* tokens,
                   int64_t N, int64_t V, int64_t D, float scale, int32_t ignore_index, void* y,
                   int32_t dtype, int64_t ldy, int32_t* status, void* stream) {
  int rc = check_embed_shape(N, V, D);
  if (rc != FLCE_OK) return rc;
  if (!known_dtype(dtype) || !known_dtype(wdtype) || !std::isfinite(scale)) return FLCE_ERR_OPTION;
  if (ldw < D || ldy < D) return FLCE_ERR_SHAPE;
  if (N == 0) return FLCE_OK;
  if (weight == nullptr || tokens == nullptr || y == nullptr) return FLCE_ERR_NULL;
  if (!aligned(weight, elem_size(wdtype)) || !aligned(y, elem_size(dtype)) || !aligned(tokens, 4) ||
      !aligned(status, 4))
    return FLCE_ERR_ALIGN;
  if (weight == y) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return launch_embedding(weight, wdtype == FLCE_DTYPE_BF16, ldw, tokens, static_cast<int>(N),
                          static_cast<int>(V), static_cast<int>(D), scale, ignore_index, y,
                          dtype == FLCE_DTYPE_BF16, ldy, status,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

int flce_embedding_backward_workspace_size(int64_t N, int64_t V, int64_t D, size_t* bytes) {
  if (bytes == nullptr) return FLCE_ERR_NULL;
  const int rc = check_embed_shape(N, V, D);
  if (rc != FLCE_OK) return rc;
  *bytes = make_embed_plan(N, D).total;
  return FLCE_OK;
}

int flce_embedding_backward(const void* dy, int32_t dtype, int64_t lddy, const int32_t* tokens,
                            int64_t N, int64_t V, int64_t D, float scale, int32_t ignore_index,
                            void* dW, int32_t wdtype, int64_t ldw, int32_t accumulate,
                            void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_embed_shape(N, V, D);
  if (rc != FLCE_OK) return rc;
  if (!known_dtype(dtype) || !known_dtype(wdtype) || !std::isfinite(scale)) return FLCE_ERR_OPTION;
  if (lddy < D || ldw < D) return FLCE_ERR_SHAPE;
  if (N == 0 && accumulate) return FLCE_OK;
  if (dW == nullptr) return FLCE_ERR_NULL;
  if (!aligned(dW, elem_size(wdtype))) return FLCE_ERR_ALIGN;
  const EmbedPlan p = make_embed_plan(N, D);
  if (N > 0) {
    if (dy == nullptr || tokens == nullptr || workspace == nullptr) return FLCE_ERR_NULL;
    if (!aligned(dy, elem_size(dtype)) || !aligned(tokens, 4) || !aligned(workspace, 16))
      return FLCE_ERR_ALIGN;
    if (dy == dW) return FLCE_ERR_OPTION;
    if (ws_bytes < p.total) return FLCE_ERR_WORKSPACE;
  }
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  auto words = [&](size_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
  uint32_t *ids = nullptr, *perm = nullptr;
  float* part = nullptr;
  if (N > 0) {
    ids = words(p.off_ids);
    perm = words(p.off_perm);
    part = reinterpret_cast<float*>(ws + p.off_part);
    if (launch_sort_tokens(tokens, static_cast<int>(N), static_cast<int>(V), ignore_index, ids, perm,
                           words(p.off_ids2), words(p.off_perm2), words(p.off_counts), st) != cudaSuccess)
      return FLCE_ERR_CUDA;
  }
  return launch_embedding_grad(dy, dtype == FLCE_DTYPE_BF16, lddy, ids, perm, static_cast<int>(N),
                               static_cast<int>(V), static_cast<int>(D), scale, dW,
                               wdtype == FLCE_DTYPE_BF16, ldw, accumulate != 0, part, st) == cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

}  // extern "C"
