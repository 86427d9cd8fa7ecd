/*
 * grad_sm103.h -- C ABI of the GB300 (sm_103a) global gradient norm over many
 * tensors, and clipping by it.
 *
 *     norm = inv_scale * sqrt(sum over tensors t, elements i of g_ti^2)
 *     out_ti = round(g_ti * inv_scale * c),  c = max_norm / norm if norm > max_norm, else 1
 *
 * inv_scale undoes a loss scale (1 where there is none).  If the norm is not
 * finite in FP32 (an infinity or NaN among the gradients, or a norm above FP32's
 * range), c = 1: the caller sees it in *norm and skips the step.
 *
 * The squares are summed in FP32 over 32 or fewer elements at a time and from
 * there on in FP64; a group of elements whose FP32 sum left the range where
 * every square is exact to FP32 (overflow, or squares that underflow) is
 * summed again in FP64, so the norm is right to a few FP32 roundings for
 * every finite input (infinity where FP32 does not hold it).  The order of the
 * sums is fixed: the same bits on every run on the same device.  FP16 and BF16
 * subnormals count.
 *
 * Tensors: `count` device pointers with their element counts and types, each
 * pointer aligned to its element size, elements contiguous; a tensor may be
 * empty.  outs[t] has the type of grads[t]; it may be grads[t] itself (in
 * place), and outs == NULL means in place for all.  In place, tensors are not
 * written when inv_scale * c is exactly 1.  max_norm = infinity (INFINITY)
 * never clips; with outs == NULL and inv_scale == 1 it only computes the norm.
 * A tensor listed twice counts twice in the norm.  Outputs that overlap each
 * other, or a gradient other than their own, are rejected (a CTA would write
 * what another still reads), and so is a tensor listed twice in place; where
 * all are in place, max_norm is infinite and inv_scale is 1, nothing but the norm
 * is written and tensors may overlap.
 *
 * The arrays grads, outs, sizes and dtypes are HOST arrays, read during the
 * call only (they travel as kernel parameters, GRAD_TENSORS_PER_LAUNCH
 * tensors per launch, so a captured graph keeps its own copy).
 *
 * `norm` (one FP32 on the device) receives the norm, and `workspace`
 * (grad_clip_workspace bytes, 16-byte aligned, contents need no preparation)
 * the partial sums; two calls that may overlap on the GPU need two of each.
 * Asynchronous on `stream`, allocates nothing, can be captured.
 *
 * Errors: GEMM_ERR_INVALID_VALUE (negative count or size, NULL or misaligned
 * pointer of a tensor that is not empty, unknown type, max_norm not positive,
 * inv_scale not positive and finite, workspace too small, overlapping
 * outputs; nothing is enqueued), GEMM_ERR_NOT_SUPPORTED (not sm_103),
 * GEMM_ERR_LAUNCH.
 */
#ifndef GRAD_SM103_H_
#define GRAD_SM103_H_

#include <stdint.h>

#include "gemm_sm103.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GRAD_TENSORS_PER_LAUNCH 512

gemm_status_t grad_clip(int64_t count, const void* const* grads, void* const* outs,
                        const int64_t* sizes, const int32_t* dtypes, float max_norm,
                        float inv_scale, float* norm, void* workspace, int64_t workspace_bytes,
                        gemm_stream_t stream);

/* Bytes of workspace for a call over `count` tensors on a device of num_sms
 * SMs (0: the current device's); -1 for bad arguments. */
int64_t grad_clip_workspace(int64_t count, int32_t num_sms);

#ifdef __cplusplus
}
#endif

#endif /* GRAD_SM103_H_ */
