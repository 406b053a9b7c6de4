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
 * are held as E4M3 codes of x / 2^e rounded to nearest even (no value saturates).
 *
 * A row of D values is a record of flce_packed_row_bytes(D) bytes, a multiple of 16:
 *   D codes, zeros up to the next multiple of 32, then one byte e + 127 per block, zeros
 *   to the record's end. Records follow one another.
 * A block that holds an infinity or a NaN has the byte 255 and stands for NaN throughout;
 * one of zeros alone has the byte 0. Values of more than 248 2^120 round to infinity.
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

#ifdef __cplusplus
}
#endif

#endif /* FLCE_BLOCKS_H_ */
