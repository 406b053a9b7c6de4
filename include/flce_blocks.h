/*
 * flce_blocks.h — C ABI of the block-scaled formats that libflce.so provides beside the
 * per-tensor E4M3 of flce.h: activations kept in 8 bits for the backward pass (alone, and
 * by the layer norm), and 4-bit floating point (quantisation, and the product of a 4-bit
 * head).
 *
 * The conventions of flce.h and flce_ops.h hold: dense row-major device memory, bf16 as
 * bit patterns, caller-owned outputs and workspaces, stream-ordered calls that allocate
 * nothing, host-side errors returned before anything is enqueued, FLCE_ERR_* codes,
 * FLCE_DTYPE_* types, strides in elements. A call with no rows is valid.
 */
#ifndef FLCE_BLOCKS_H_
#define FLCE_BLOCKS_H_

#include <stddef.h>
#include <stdint.h>

#include "flce.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * 8 bits: each 32 values of a row (the last block may be shorter) have a scale 2^e, e the
 * smallest integer >= -127 for which the block's largest magnitude is at most 448 2^e, and
 * are held as E4M3 codes of x / 2^e rounded to nearest even (no value saturates, where the
 * rounding down of e that the microscaling standard describes lets the largest ones).
 *
 * A row of D values is a record of flce_packed_row_bytes(D) bytes, a multiple of 16:
 *   D codes, zeros up to the next multiple of 32, then one byte e + 127 per block, zeros
 *   to the record's end. Records follow one another.
 * A block that holds an infinity or a NaN has the byte 255 and stands for NaN throughout;
 * one of zeros alone has the byte 0. Values of 248 2^120 and more stand for infinity.
 */
int flce_packed_row_bytes(int64_t D, int64_t* bytes);

/* x [N, D] of dtype, row stride ldx >= D, aligned to its element size; packed: N records,
 * 16-byte aligned. */
int flce_pack_e4m3(const void* x, int32_t dtype, int64_t ldx, int64_t N, int64_t D,
                   uint8_t* packed, void* stream);

/* The values that the records stand for, rounded once to dtype (exact in fp32 and bf16 but
 * for what is below their smallest normal number). */
int flce_unpack_e4m3(const uint8_t* packed, int64_t N, int64_t D, void* x, int32_t dtype,
                     int64_t ldx, void* stream);

/*
 * flce_layer_norm (flce_ops.h) that also leaves its input packed, and the gradients from
 * that instead of from x: with x~ the values that the records stand for and mean, rstd
 * those of x itself, h = (x~ - mean) rstd takes h's place in flce_layer_norm_backward's
 * formulas. What is kept between the two calls is 1.03 bytes a value.
 *
 * Arguments as in flce_ops.h; packed as above. y may be x. workspace: as
 * flce_layer_norm_workspace_size() has it.
 */
int flce_layer_norm_packed(const void* x, int32_t dtype, int64_t ldx, const void* weight,
                           const void* bias, int32_t wdtype, int64_t N, int64_t D, float eps,
                           void* y, int64_t ldy, float* mean, float* rstd, uint8_t* packed,
                           void* stream);
int flce_layer_norm_packed_backward(const void* dy, int32_t dtype, int64_t lddy,
                                    const uint8_t* packed, const void* weight, int32_t wdtype,
                                    const float* mean, const float* rstd, int64_t N, int64_t D,
                                    void* dx, int64_t lddx, void* dweight, void* dbias,
                                    void* workspace, size_t ws_bytes, void* stream);

/*
 * 4-bit floating point: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with a
 * scale for each block of neighbouring values of a row (the last block may be shorter).
 *
 *   FLCE_FP4_MX   blocks of 32, scale 2^e, e the smallest integer >= -127 for which the
 *                 block's largest magnitude is at most 6 2^e; code rn(x / 2^e)
 *   FLCE_FP4_NV   blocks of 16, an E4M3 scale s and an fp32 scale g of the row: g the
 *                 smallest power of two >= 2^-126 for which the row's largest finite
 *                 magnitude is at most 6 448 g (1 for a row of zeros), s = rn(largest
 *                 magnitude of the block / 6 / g), code rn(x / (s g)), 0 where s is 0
 *
 * All rounded to nearest even, once; a code is at most 6. A block that holds an infinity or
 * a NaN has the scale NaN (byte 255, 127) and the codes 0: it stands for NaN throughout.
 * What a block of the largest fp32 numbers stands for may be past them: infinity.
 *
 * Where the usual rules differ: the microscaling standard rounds e down, so that a block's
 * largest values may saturate, here up; nvfp4 elsewhere has one fp32 number g for the tensor.
 * Such matrices are decoded and multiplied all the same: any bytes e + 127, any E4M3 scales
 * without a sign (bytes 0 to 127), any fp32 row scales.
 *
 * Three arrays hold [N, D] (flce_fp4_sizes gives the bytes; 16-byte aligned but for
 * row_scales, 4):
 *   codes       a row in code_row_bytes: two codes to a byte, the first in the low bits,
 *               zeros up to the next multiple of 64 values
 *   scales      bytes (e + 127, or E4M3 codes) in groups of 512: for 128 rows and 4
 *               neighbouring blocks, row r's four bytes at (r % 32) 16 + (r / 32) 4. Blocks
 *               are padded with zeros to whole 256 values, rows to whole 128s; the groups
 *               of 128 rows follow one another
 *   row_scales  fp32 [N] (FLCE_FP4_NV; NULL otherwise)
 */
enum { FLCE_FP4_MX = 0, FLCE_FP4_NV = 1 };
int flce_fp4_sizes(int64_t N, int64_t D, int32_t format, int64_t* code_row_bytes,
                   size_t* scale_bytes);

/* x [N, D] of dtype, row stride ldx >= D, aligned to its element size. */
int flce_quantize_fp4(const void* x, int32_t dtype, int64_t ldx, int64_t N, int64_t D,
                      int32_t format, uint8_t* codes, uint8_t* scales, float* row_scales,
                      void* stream);

/* The values, code scale row_scale in fp32, rounded once to dtype. */
int flce_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* row_scales,
                        int64_t N, int64_t D, int32_t format, void* x, int32_t dtype,
                        int64_t ldx, void* stream);

/*
 * y = H W^T of two such matrices of one format, H [N, D] (tokens) and W [V, D] (a head or
 * another linear layer's weight), on the block-scaled tensor cores: the blocks' products
 * are accumulated in fp32, multiplied in fp32 by W's row scale and then by H's, and rounded
 * once to dtype.
 *   y        [N, V] of dtype (FLCE_DTYPE_F32 / _BF16), row stride ldy >= V, aligned to its
 *            element size
 *   timeout_ns  limit of every device-side wait; 0 = 2 s
 *   status   int32 [1] or NULL; written only when the device finds an error: a wait that
 *            ran out of time gives FLCE_ERR_TIMEOUT and NaN for what was not done
 * Results do not change from run to run, and a token's do not depend on the others'.
 */
int flce_linear_fp4(const uint8_t* h_codes, const uint8_t* h_scales, const float* h_row_scales,
                    const uint8_t* w_codes, const uint8_t* w_scales, const float* w_row_scales,
                    int64_t N, int64_t D, int64_t V, int32_t format, void* y, int32_t dtype,
                    int64_t ldy, int64_t timeout_ns, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_BLOCKS_H_ */
