/*
 * expert_sm103.h -- C ABI of the GB300 (sm_103a) row moves around a feed-forward
 * block with experts: tokens sorted by expert, their rows brought together and
 * back with the router's weights applied, and the backward passes of both moves.
 *
 * A token t has k choices, slots s = t k + j, each an expert's number or none.
 *
 *   expert_sort:     order = the slots that chose an expert, by expert, and by slot
 *                    within an expert; pos[order[i]] = i; offsets[e] = slots of
 *                    experts below e (so expert e has rows offsets[e] ..
 *                    offsets[e + 1] - 1)
 *   expert_gather:   Xs[pos[t,j]] = round(w[t,j] X[t])
 *   expert_combine:  Y[t] = round(sum over j of w[t,j] Ys[pos[t,j]])
 *   expert_gather_backward, from dXs:
 *                    dX[t] = round(sum over j of w[t,j] dXs[pos[t,j]])
 *                    dw[t,j] = round(X[t] . dXs[pos[t,j]])
 *   expert_combine_backward, from dY:
 *                    dYs[pos[t,j]] = round(w[t,j] dY[t])
 *                    dw[t,j] = round(dY[t] . Ys[pos[t,j]])
 *
 * Products and sums are FP32 (j upwards; a dot product in an order that depends on
 * sizes and alignment alone), each result rounded once.  weight == NULL: every weight is
 * 1.  A slot that chose no expert (its id outside 0 .. E - 1; its position -1)
 * takes no part: nothing of it is read or written but dw = 0, and a token with no
 * choices left has Y = 0.  Otherwise IEEE arithmetic (a weight of 0 times an
 * infinity gives NaN).
 *
 * Matrices are row-major with leading dimensions in elements, at least the row
 * length; every pointer is aligned to its element size.  X, Y, dX, dY (T x D) and
 * Xs, Ys, dXs, dYs (rows x D) share one type, F16, BF16 or F32; weight and dweight
 * (T x k) have one each of these.  pos is T x k without padding, order has T k
 * elements (-1 from offsets[E] on), both int32; ids are int32 or int64.  Rows of
 * Xs and dYs that no position names, and padding columns, are left as they were.
 * A position outside 0 .. rows - 1 counts as none.
 *
 * Positions that are not -1 must differ where rows are written (as expert_sort's
 * do).  Outputs must not overlap inputs or each other, element by element (columns of one
 * buffer are apart), but for dYs, which may be Ys (same leading dimension).
 *
 * No handle and no workspace: asynchronous on `stream`, nothing allocated, can be
 * captured.  The same call gives the same bits.
 *
 * Errors: GEMM_ERR_INVALID_VALUE (a negative size, T k, D or rows
 * above 2^30, E below 1 or
 * above EXPERT_MAX, a leading dimension below its row's length, an unknown type,
 * NULL or misaligned pointers of what is not empty, overlap; nothing is enqueued),
 * GEMM_ERR_NOT_SUPPORTED (not sm_103), GEMM_ERR_LAUNCH.
 */
#ifndef EXPERT_SM103_H_
#define EXPERT_SM103_H_

#include <stdint.h>

#include "gemm_sm103.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EXPERT_MAX 1024

/* ids: T x k, id_bytes 4 or 8 each.  order may be NULL (not wanted). */
gemm_status_t expert_sort(int64_t T, int64_t k, int64_t E, const void* ids, int64_t ldids,
                          int32_t id_bytes, int32_t* pos, int32_t* offsets, int32_t* order,
                          gemm_stream_t stream);

typedef struct {
    const void* weight;    /* device, T x k, or NULL: all 1 */
    int64_t ldw;
    int32_t weight_dtype;
    void* dweight;         /* device, T x k, or NULL: not wanted (backward passes only) */
    int64_t lddw;
    int32_t dweight_dtype;
} expert_weights_t;

/* w may be NULL (no weights). */
gemm_status_t expert_gather(int64_t T, int64_t k, int64_t D, int64_t rows, const void* X,
                            int64_t ldx, const int32_t* pos, void* Xs, int64_t ldxs,
                            int32_t dtype, const expert_weights_t* w, gemm_stream_t stream);

gemm_status_t expert_combine(int64_t T, int64_t k, int64_t D, int64_t rows, const void* Ys,
                             int64_t ldys, const int32_t* pos, void* Y, int64_t ldy,
                             int32_t dtype, const expert_weights_t* w, gemm_stream_t stream);

/* dX may be NULL (not wanted); X may be NULL without dweight. */
gemm_status_t expert_gather_backward(int64_t T, int64_t k, int64_t D, int64_t rows,
                                     const void* dXs, int64_t lddxs, const void* X, int64_t ldx,
                                     const int32_t* pos, void* dX, int64_t lddx, int32_t dtype,
                                     const expert_weights_t* w, gemm_stream_t stream);

/* dYs may be NULL (not wanted); Ys may be NULL without dweight. */
gemm_status_t expert_combine_backward(int64_t T, int64_t k, int64_t D, int64_t rows,
                                      const void* dY, int64_t lddy, const void* Ys, int64_t ldys,
                                      const int32_t* pos, void* dYs, int64_t lddys, int32_t dtype,
                                      const expert_weights_t* w, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EXPERT_SM103_H_ */
