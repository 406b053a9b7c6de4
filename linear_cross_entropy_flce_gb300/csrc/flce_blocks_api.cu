// C ABI of the block-scaled formats (declared in include/flce_blocks.h): argument checks and launch
// sequences.
//
//   flce_pack_e4m3, flce_unpack_e4m3   one kernel
//   flce_layer_norm_packed             the pack of x, then flce_layer_norm
//   flce_layer_norm_packed_backward    as flce_layer_norm_backward
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/flce_blocks.h"
#include "../../include/flce_ops.h"
#include "flce_blocks.h"
#include "flce_host.h"

namespace flce {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t elem_size(int32_t dtype) { return dtype == FLCE_DTYPE_BF16 ? 2 : 4; }
bool known_dtype(int32_t dtype) { return dtype == FLCE_DTYPE_F32 || dtype == FLCE_DTYPE_BF16; }

int check_matrix(int64_t N, int64_t D, int32_t dtype, int64_t ld) {
  if (N < 0 || N > (int64_t(1) << 30) || D < 1 || D > (int64_t(1) << 24)) return FLCE_ERR_SHAPE;
  if (!known_dtype(dtype)) return FLCE_ERR_OPTION;
  return ld < D ? FLCE_ERR_SHAPE : FLCE_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA; }

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_packed_row_bytes(int64_t D, int64_t* bytes) {
  if (bytes == nullptr) return FLCE_ERR_NULL;
  if (D < 1 || D > (int64_t(1) << 24)) return FLCE_ERR_SHAPE;
  *bytes = packed_record(D);
  return FLCE_OK;
}

int flce_pack_e4m3(const void* x, int32_t dtype, int64_t ldx, int64_t N, int64_t D,
                   uint8_t* packed, void* stream) {
  int rc = check_matrix(N, D, dtype, ldx);
  if (rc != FLCE_OK || N == 0) return rc;
  if (x == nullptr || packed == nullptr) return FLCE_ERR_NULL;
  if (!aligned(x, elem_size(dtype)) || !aligned(packed, 16)) return FLCE_ERR_ALIGN;
  if (x == packed) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return done(launch_pack_e4m3(x, dtype == FLCE_DTYPE_BF16, ldx, static_cast<int>(N), static_cast<int>(D),
                               packed, static_cast<cudaStream_t>(stream)));
}

int flce_unpack_e4m3(const uint8_t* packed, int64_t N, int64_t D, void* x, int32_t dtype,
                     int64_t ldx, void* stream) {
  int rc = check_matrix(N, D, dtype, ldx);
  if (rc != FLCE_OK || N == 0) return rc;
  if (x == nullptr || packed == nullptr) return FLCE_ERR_NULL;
  if (!aligned(x, elem_size(dtype)) || !aligned(packed, 16)) return FLCE_ERR_ALIGN;
  if (x == packed) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return done(launch_unpack_e4m3(packed, static_cast<int>(N), static_cast<int>(D), x, dtype == FLCE_DTYPE_BF16,
                                 ldx, static_cast<cudaStream_t>(stream)));
}

int flce_layer_norm_packed(const void* x, int32_t dtype, int64_t ldx, const void* weight,
                           const void* bias, int32_t wdtype, int64_t N, int64_t D, float eps,
                           void* y, int64_t ldy, float* mean, float* rstd, uint8_t* packed,
                           void* stream) {
  // what flce_layer_norm refuses is refused before the pack is enqueued
  int rc = check_matrix(N, D, dtype, ldx);
  if (rc != FLCE_OK) return rc;
  if (!known_dtype(wdtype) || !(eps >= 0.f) || std::isinf(eps)) return FLCE_ERR_OPTION;
  if (ldy < D) return FLCE_ERR_SHAPE;
  if (N == 0) return FLCE_OK;
  if (x == nullptr || y == nullptr || packed == nullptr) return FLCE_ERR_NULL;
  const size_t e = elem_size(dtype), ew = elem_size(wdtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(weight, ew) || !aligned(bias, ew) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(packed, 16))
    return FLCE_ERR_ALIGN;
  if ((x == y && ldx != ldy) || packed == x || packed == y) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_pack_e4m3(x, dtype == FLCE_DTYPE_BF16, ldx, static_cast<int>(N), static_cast<int>(D), packed, st) !=
      cudaSuccess)
    return FLCE_ERR_CUDA;
  return done(launch_layer_norm(x, dtype == FLCE_DTYPE_BF16, ldx, weight, bias, wdtype == FLCE_DTYPE_BF16,
                                static_cast<int>(N), static_cast<int>(D), eps, y, ldy, mean, rstd, sms, st));
}

int flce_layer_norm_packed_backward(const void* dy, int32_t dtype, int64_t lddy,
                                    const uint8_t* packed, const void* weight, int32_t wdtype,
                                    const float* mean, const float* rstd, int64_t N, int64_t D,
                                    void* dx, int64_t lddx, void* dweight, void* dbias,
                                    void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_matrix(N, D, dtype, lddy);
  if (rc != FLCE_OK) return rc;
  if (!known_dtype(wdtype)) return FLCE_ERR_OPTION;
  if (dx != nullptr && lddx < D) return FLCE_ERR_SHAPE;
  const bool columns = dweight != nullptr || dbias != nullptr;
  if (N == 0 && !columns) return FLCE_OK;
  const size_t e = elem_size(dtype), ew = elem_size(wdtype);
  if (N > 0) {
    if (dy == nullptr || packed == nullptr || mean == nullptr || rstd == nullptr ||
        (columns && workspace == nullptr))
      return FLCE_ERR_NULL;
    size_t need = 0;
    rc = flce_layer_norm_workspace_size(N, D, &need);
    if (rc != FLCE_OK) return rc;
    if (columns && ws_bytes < need) return FLCE_ERR_WORKSPACE;
  }
  if (!aligned(dy, e) || !aligned(packed, 16) || !aligned(dx, e) || !aligned(weight, ew) ||
      !aligned(dweight, ew) || !aligned(dbias, ew) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(workspace, 16))
    return FLCE_ERR_ALIGN;
  if (dx != nullptr && ((dx == dy && lddx != lddy) || dx == packed)) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return done(launch_layer_norm_backward_packed(dy, lddy, packed, dtype == FLCE_DTYPE_BF16, weight,
                                                wdtype == FLCE_DTYPE_BF16, mean, rstd, static_cast<int>(N),
                                                static_cast<int>(D), dx, lddx, dweight, dbias,
                                                static_cast<float*>(workspace), sms,
                                                static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
