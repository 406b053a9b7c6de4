// C ABI of the block-scaled formats (declared in include/flce_blocks.h): argument checks and launch
// sequences.
//
//   flce_pack_e4m3, flce_unpack_e4m3   one kernel
//   flce_layer_norm_packed             one kernel; rows that no CTA holds: the pack of x, then
//                                      flce_layer_norm's
//   flce_layer_norm_packed_backward    as flce_layer_norm_backward
//   flce_quantize_fp4, flce_dequantize_fp4, flce_linear_fp4   one kernel
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/flce_blocks.h"
#include "../../include/flce_ops.h"
#include "flce_blocks.h"
#include "flce_fp4_gemm.h"
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

int check_fp4(int64_t N, int64_t D, int32_t format) {
  if (N < 0 || N > (int64_t(1) << 30) || D < 1 || D > (int64_t(1) << 24)) return FLCE_ERR_SHAPE;
  return format == FLCE_FP4_MX || format == FLCE_FP4_NV ? FLCE_OK : FLCE_ERR_OPTION;
}

// A matrix's three arrays.
int check_fp4_arrays(const uint8_t* codes, const uint8_t* scales, const float* row_scales, int32_t format) {
  if (codes == nullptr || scales == nullptr || (format == FLCE_FP4_NV && row_scales == nullptr))
    return FLCE_ERR_NULL;
  return aligned(codes, 16) && aligned(scales, 16) && aligned(row_scales, 4) ? FLCE_OK : FLCE_ERR_ALIGN;
}

// Codes [rows][row_bytes] in boxes of 128 bytes x box_rows with 128-byte swizzle; what is outside reads as
// zero.
bool encode_codes(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {row_bytes, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Groups of 512 scale bytes, in boxes of those of 128 rows' 256 values; none past the last reads as zero.
bool encode_scales(CUtensorMap* m, const void* base, uint64_t bytes, int nv) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {128, bytes / 512};
  cuuint64_t strides[1] = {512};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(fp4_stage_scales(nv) / 512)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y in boxes of 32 values of kFp4OutTokens rows; nothing outside y is written.
bool encode_y(CUtensorMap* m, void* y, int64_t V, int64_t N, int64_t ldy) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(V), static_cast<cuuint64_t>(N)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldy) * 2};
  cuuint32_t box[2] = {32, kFp4OutTokens};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
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
  return done(launch_layer_norm_packed(x, dtype == FLCE_DTYPE_BF16, ldx, weight, bias, wdtype == FLCE_DTYPE_BF16,
                                       static_cast<int>(N), static_cast<int>(D), eps, y, ldy, mean, rstd, packed,
                                       sms, static_cast<cudaStream_t>(stream)));
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

int flce_fp4_sizes(int64_t N, int64_t D, int32_t format, int64_t* code_row_bytes, size_t* scale_bytes) {
  if (code_row_bytes == nullptr || scale_bytes == nullptr) return FLCE_ERR_NULL;
  const int rc = check_fp4(N, D, format);
  if (rc != FLCE_OK) return rc;
  *code_row_bytes = fp4_code_bytes(D);
  *scale_bytes = static_cast<size_t>(fp4_scale_bytes(N, D, format == FLCE_FP4_NV));
  return FLCE_OK;
}

int flce_quantize_fp4(const void* x, int32_t dtype, int64_t ldx, int64_t N, int64_t D, int32_t format,
                      uint8_t* codes, uint8_t* scales, float* row_scales, void* stream) {
  int rc = check_matrix(N, D, dtype, ldx);
  if (rc == FLCE_OK) rc = check_fp4(N, D, format);
  if (rc != FLCE_OK || N == 0) return rc;
  if (x == nullptr) return FLCE_ERR_NULL;
  rc = check_fp4_arrays(codes, scales, row_scales, format);
  if (rc != FLCE_OK) return rc;
  if (!aligned(x, elem_size(dtype))) return FLCE_ERR_ALIGN;
  if (x == codes || x == scales || codes == scales) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return done(launch_quantize_fp4(x, dtype == FLCE_DTYPE_BF16, ldx, static_cast<int>(N), static_cast<int>(D),
                                  format == FLCE_FP4_NV, codes, scales, row_scales,
                                  static_cast<cudaStream_t>(stream)));
}

int flce_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* row_scales, int64_t N,
                        int64_t D, int32_t format, void* x, int32_t dtype, int64_t ldx, void* stream) {
  int rc = check_matrix(N, D, dtype, ldx);
  if (rc == FLCE_OK) rc = check_fp4(N, D, format);
  if (rc != FLCE_OK || N == 0) return rc;
  if (x == nullptr) return FLCE_ERR_NULL;
  rc = check_fp4_arrays(codes, scales, row_scales, format);
  if (rc != FLCE_OK) return rc;
  if (!aligned(x, elem_size(dtype))) return FLCE_ERR_ALIGN;
  if (x == codes || x == scales) return FLCE_ERR_OPTION;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return done(launch_dequantize_fp4(codes, scales, row_scales, static_cast<int>(N), static_cast<int>(D),
                                    format == FLCE_FP4_NV, x, dtype == FLCE_DTYPE_BF16, ldx,
                                    static_cast<cudaStream_t>(stream)));
}

int flce_linear_fp4(const uint8_t* h_codes, const uint8_t* h_scales, const float* h_row_scales,
                    const uint8_t* w_codes, const uint8_t* w_scales, const float* w_row_scales, int64_t N,
                    int64_t D, int64_t V, int32_t format, void* y, int32_t dtype, int64_t ldy,
                    int64_t timeout_ns, int32_t* status, void* stream) {
  int rc = check_fp4(N, D, format);
  if (rc != FLCE_OK) return rc;
  if (V < 1 || V > (int64_t(1) << 30) || ldy < V) return FLCE_ERR_SHAPE;
  if (!known_dtype(dtype) || timeout_ns < 0) return FLCE_ERR_OPTION;
  if (N == 0) return FLCE_OK;
  rc = check_fp4_arrays(h_codes, h_scales, h_row_scales, format);
  if (rc == FLCE_OK) rc = check_fp4_arrays(w_codes, w_scales, w_row_scales, format);
  if (rc != FLCE_OK) return rc;
  if (y == nullptr) return FLCE_ERR_NULL;
  if (!aligned(y, elem_size(dtype)) || !aligned(status, 4)) return FLCE_ERR_ALIGN;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  Fp4Maps maps{};
  const int bf16 = dtype == FLCE_DTYPE_BF16;
  const int nv = format == FLCE_FP4_NV;
  const bool boxes = fp4_boxes(fp4_tile(N), bf16) && aligned(y, 16) && ldy % 8 == 0 && encode_y(&maps.y, y, V, N, ldy);
  const int kn = boxes ? fp4_wide_tile(N, V, sms, nv) : fp4_tile(N);
  const uint64_t row = static_cast<uint64_t>(fp4_code_bytes(D));
  if (!encode_codes(&maps.w, w_codes, row, static_cast<uint64_t>(V), 128) ||
      !encode_codes(&maps.w32, w_codes, row, static_cast<uint64_t>(V), 32) ||
      !encode_codes(&maps.h, h_codes, row, static_cast<uint64_t>(N), kn > 256 ? 64u : static_cast<uint32_t>(kn / fp4_ctas(kn))) ||
      !encode_scales(&maps.w_scales, w_scales, static_cast<uint64_t>(fp4_scale_bytes(V, D, nv)), nv) ||
      !encode_scales(&maps.h_scales, h_scales, static_cast<uint64_t>(fp4_scale_bytes(N, D, nv)), nv))
    return FLCE_ERR_CUDA;
  Fp4GemmParams p{};
  p.N = static_cast<int>(N);
  p.V = static_cast<int>(V);
  p.stages = static_cast<int>(fp4_stages(D));
  p.h_rows = h_row_scales;
  p.w_rows = w_row_scales;
  p.y = y;
  p.ldy = ldy;
  p.wide = boxes;
  p.timeout_ns = timeout_ns > 0 ? timeout_ns : kDefaultTimeoutNs;
  p.status = status;
  return done(launch_fp4_gemm(kn, nv, bf16, maps, p, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
