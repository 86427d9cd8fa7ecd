/*
 * norm_sm103.h -- C ABI of the GB300 (sm_103a) norms before and after a
 * transformer block, fused with the block's gate, its residual scale and the
 * residual add.
 *
 * One pass over the rows joins a block's output Z (M x N) to the residual
 * stream X (M x N) and normalises the result for the next block:
 *     n_ij  = Norm_post(Z_i)_j * post_weight_j + post_bias_j
 *     XO_ij = round_X(X_ij + scale * gate_{i / gate_rows, j} * n_ij)
 *     Y_ij  = round_Z(Norm_pre(XO_i)_j * pre_weight_j + pre_bias_j)
 * Norm along a row v of N elements is one of
 *     NORM_NONE   v
 *     NORM_RMS    v / sqrt(mean(v^2) + eps)
 *     NORM_LAYER  (v - mean(v)) / sqrt(var(v) + eps), var the biased variance
 * with the statistics in FP32 (the variance from the deviations about the
 * mean).  Everything is FP32 between the loads and the one rounding of each
 * result; Norm_pre sees XO as its type holds it, so that the backward pass,
 * which reads the stored XO, differentiates what was computed.
 *
 * Optional parts: Z NULL skips the first two lines (Y = Norm_pre(X); XO must
 * be NULL); Y NULL skips the last.  NULL weights and gate read as 1, NULL
 * biases as 0.  post NORM_NONE with weights is an affine of Z.
 *
 * The gate has ceil(M / gate_rows) rows of N elements, ld_gate apart: one row
 * for all of X (gate_rows >= M: a scale per channel), one per sequence
 * (gate_rows = its tokens) or one per token (gate_rows = 1).
 *
 * Backward.  Given the loss's gradients dY (with respect to Y) and dXO (with
 * respect to XO from everything else that reads it):
 *     dXO'  = dXO + J_pre(XO_i)^T (dY * pre_weight)
 *     dX    = round_X(dXO')
 *     dn    = scale * gate * dXO'
 *     dZ    = round_Z(J_post(Z_i)^T (dn * post_weight))
 *     d_pre_weight_j  = sum_i dY_ij Norm_pre(XO_i)_j     d_pre_bias_j  = sum_i dY_ij
 *     d_post_weight_j = sum_i dn_ij Norm_post(Z_i)_j     d_post_bias_j = sum_i dn_ij
 *     d_gate_gj       = scale * sum over the rows i of group g of dXO'_ij n_ij
 * J the Jacobian of the norm.  The statistics are computed again from XO and
 * Z; nothing else is kept from the forward pass.  dY NULL (and dXO NULL) read
 * as 0; every output may be NULL (not wanted).  The sums over rows are FP32
 * partial sums per CTA, added in a fixed order: the same bits on every run.
 *
 * Layout: row-major, element (i, j) of a matrix at i * ld + j, unit stride in
 * j, any ld >= N; every pointer aligned to its element size.  Columns j >= N
 * of a row are never touched.  X, XO, dX, dXO share x_dtype; Z, Y, dZ, dY
 * share z_dtype; (x_dtype, z_dtype) is one of (F16, F16), (BF16, BF16),
 * (F32, F32), (F32, F16), (F32, BF16).  Weights, biases and the gate share
 * vec_dtype, their gradients grad_dtype (F16, BF16 or F32).
 * N is at most NORM_MAX_N (NOT_SUPPORTED beyond); M is any.
 *
 * XO may be X itself, dX may be dXO itself, dZ may be Z, and Y or dY's
 * storage may be reused only after the call: any other overlap of an output
 * with an input or another output gives undefined values.
 *
 * Ownership and threading: DEVICE pointers of the caller, on the current
 * device; the calls are asynchronous on `stream`, allocate nothing and keep
 * nothing.  The backward pass writes its partial sums to the caller's
 * workspace (norm_block_backward_workspace bytes, 16-byte aligned; its
 * contents need no preparation): 16 N bytes for each chunk of rows, of which
 * there are about as many as SMs but at least one for every group of the gate.
 * With 1 < gate_rows < M that is at least 16 N ceil(M / gate_rows) bytes, for
 * two rows per group and 16-bit rows four times the size of X.  Two calls that
 * may overlap on the GPU need two workspaces.  Both calls can be captured into a CUDA graph.
 *
 * Errors: GEMM_ERR_INVALID_VALUE (bad size, leading dimension, type, kind,
 * NULL or misaligned pointer, eps not positive and finite, scale not finite,
 * workspace too small; nothing is enqueued), GEMM_ERR_NOT_SUPPORTED (N too
 * large, a pair of types not listed, or the device is not sm_103),
 * GEMM_ERR_LAUNCH.
 */
#ifndef NORM_SM103_H_
#define NORM_SM103_H_

#include <stdint.h>

#include "gemm_sm103.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NORM_MAX_N 16384

typedef enum { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 } norm_kind_t;

/* The norms, weights and gate of a block (what a model keeps). */
typedef struct {
    int32_t pre, post;         /* norm_kind_t */
    const void* pre_weight;    /* N elements or NULL (1) */
    const void* pre_bias;      /* N elements or NULL (0) */
    const void* post_weight;
    const void* post_bias;
    const void* gate;          /* ceil(M / gate_rows) x N, or NULL (1) */
    int64_t ld_gate;           /* elements between the gate's rows (>= N) */
    int64_t gate_rows;         /* rows of X that share a row of the gate (>= 1) */
    int32_t vec_dtype;         /* type of the weights, biases and gate */
    float scale;               /* residual scale */
    float eps;                 /* > 0 */
} norm_block_t;

/* The gradients of the weights, biases and gate, each NULL if not wanted. */
typedef struct {
    void* d_pre_weight;
    void* d_pre_bias;
    void* d_post_weight;
    void* d_post_bias;
    void* d_gate;              /* as the gate, tightly packed (row pitch N) */
    int32_t grad_dtype;
} norm_block_grads_t;

/* XO = X + scale * gate * Norm_post(Z), Y = Norm_pre(XO); see above. */
gemm_status_t norm_block_forward(int64_t M, int64_t N, const void* X, int64_t ldx,
                                 const void* Z, int64_t ldz, void* XO, int64_t ldxo,
                                 void* Y, int64_t ldy, int32_t x_dtype, int32_t z_dtype,
                                 const norm_block_t* block, gemm_stream_t stream);

/*
 * The backward pass.  XO: the stored output of the forward pass (X where Z is
 * NULL).  Z, dZ, d_post_* and d_gate go with Z != NULL.  With Z NULL,
 * dX = dXO + J_pre^T (dY * pre_weight).
 */
gemm_status_t norm_block_backward(int64_t M, int64_t N, const void* XO, int64_t ldxo,
                                  const void* Z, int64_t ldz, const void* dY, int64_t lddy,
                                  const void* dXO, int64_t lddxo, void* dX, int64_t lddx,
                                  void* dZ, int64_t lddz, int32_t x_dtype, int32_t z_dtype,
                                  const norm_block_t* block, const norm_block_grads_t* grads,
                                  void* workspace, int64_t workspace_bytes,
                                  gemm_stream_t stream);

/* Bytes of workspace norm_block_backward needs for M x N rows and a gate of
 * gate_rows (pass M, or 1, where there is no gate) on a device of num_sms SMs
 * (0: the current device's); -1 for bad arguments.  Host logic only when
 * num_sms > 0. */
int64_t norm_block_backward_workspace(int64_t M, int64_t N, int64_t gate_rows, int32_t num_sms);

#ifdef __cplusplus
}
#endif

#endif /* NORM_SM103_H_ */
