/*
 * flce_embed.h — C ABI of the embedding lookup that libflce.so provides next to the
 * head (flce.h): the other end of a table that the two share, and its gradient, which
 * can be added to the dW that the head's calls leave.
 *
 * The conventions of flce.h and flce_ops.h hold: dense row-major device memory, bf16 as
 * bit patterns, caller-owned outputs and workspaces, stream-ordered calls that allocate
 * nothing, host-side errors returned before anything is enqueued, FLCE_ERR_* codes,
 * FLCE_DTYPE_* types, strides in elements.
 */
#ifndef FLCE_EMBED_H_
#define FLCE_EMBED_H_

#include <stddef.h>
#include <stdint.h>

#include "flce.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * y_n = scale W[tokens_n]
 *
 *   weight   [V, D] of wdtype (FLCE_DTYPE_F32 / _BF16), row stride ldw >= D
 *   tokens   int32 [N], 4-byte aligned: ids in [0, V) or ignore_index, whose rows are 0
 *   y        [N, D] of dtype, row stride ldy >= D; must not overlap weight
 *   status   int32 [1] or NULL; written only when the device finds an error
 * Products are fp32, rounded once to dtype. A token outside [0, V) that is not
 * ignore_index gives a row of NaN and FLCE_ERR_LABEL_RANGE. Every pointer is aligned to
 * its element size (rows of whole 16 bytes are fastest); scale is finite. N = 0 is valid.
 */
int flce_embedding(const void* weight, int32_t wdtype, int64_t ldw, const int32_t* tokens,
                   int64_t N, int64_t V, int64_t D, float scale, int32_t ignore_index, void* y,
                   int32_t dtype, int64_t ldy, int32_t* status, void* stream);

/*
 * Its gradient in the table: with g_v = scale sum_{n: tokens_n = v} dy_n,
 *
 *   accumulate = 0: dW[v] = g_v for every v in [0, V) (0 for ids without tokens)
 *   accumulate = 1: dW[v] += g_v for the ids that have tokens; no other row is read or
 *                   written
 *
 *   dy   [N, D] of dtype, row stride lddy >= D
 *   dW   [V, D] of wdtype, row stride ldw >= D; must not overlap dy
 * Tokens are sorted by id, stably, and each row's sum runs over them in that order in
 * fp32, split only where the sorted order is cut into equal ranges: results do not
 * change from run to run. The sum (and, accumulating, its sum with the old value) is
 * rounded once. Tokens outside [0, V), ignore_index among them, count nowhere.
 * workspace (16-byte aligned): flce_embedding_backward_workspace_size() bytes.
 */
int flce_embedding_backward_workspace_size(int64_t N, int64_t V, int64_t D, size_t* bytes);
int flce_embedding_backward(const void* dy, int32_t dtype, int64_t lddy, const int32_t* tokens,
                            int64_t N, int64_t V, int64_t D, float scale, int32_t ignore_index,
                            void* dW, int32_t wdtype, int64_t ldw, int32_t accumulate,
                            void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_EMBED_H_ */
