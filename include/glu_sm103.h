/*
 * glu_sm103.h -- C ABI of the GB300 (sm_103a) gated linear layer (the first
 * half of a gated feed-forward block) and its backward pass.
 *
 * With X (M x K) the input, W (2F x K) the weights -- the gate's F rows, then
 * the up projection's F rows -- and an optional bias of 2F elements:
 *     P = X W^T + bias                (M x 2F: columns 0..F-1 the gate's G, F..2F-1 U)
 *     H = act(G) * U                  (M x F)
 * Both projections, the activation and the product run in one kernel (behind
 * copies of rows that are not 16-byte aligned): G and U of an output element are
 * accumulated in FP32, and H is rounded once.  In general that is the GEMM's
 * tcgen05 kernel on its own tile schedules (CTA pairs, single CTAs, stream-K,
 * swapped tiles), with G and U of a tile side by side in tensor memory; up to 128
 * rows go to a tcgen05 kernel that streams W where few tiles make it the faster
 * one, and 1 or 2 aligned rows to FP32 dot products.  P is written (rounded once,
 * from the same FP32 values) where the caller asks for it, for the backward pass.
 *
 * act is any gemm_activation_t, with the accuracy stated there.  act(G) * U
 * follows IEEE arithmetic (0 * inf and NaN give NaN).
 *
 * Backward.  Given dH (M x F) and the stored P:
 *     dG = dH * U * act'(G),  dU = dH * act(G)      dP = [dG dU]   (M x 2F)
 *     dX = dP W                                     (M x K)
 *     dW = dP^T X + beta_w * dW                     (2F x K)
 *     dbias = column sums of dP                     (2F)
 * dP is rounded to the inputs' type before the two products (the tensor core
 * reads 16-bit operands); dbias sums the unrounded FP32 values, in a fixed
 * order.  ReLU'(x) is 1 for x > 0 and 0 otherwise.
 *
 * Layout: row-major with leading dimensions in elements; every pointer
 * aligned to its element size; any leading dimension >= the row length (rows
 * that are not 16-byte aligned are copied to the handle's workspace first).
 * Padding columns are never touched.  Outputs must not overlap inputs or each
 * other, but for dP, which may be P.
 *
 * Types: X, W, dH and dP are F16 or BF16, all the same; H and P share a type,
 * dX and dW have one each (F16, BF16 or F32).  FP32 (TF32) inputs return
 * NOT_SUPPORTED.
 *
 * Ownership, threading, workspace and errors: as gemm_run (gemm_sm103.h), on the
 * handle's device, which has to be current (INVALID_VALUE otherwise): the
 * handle's workspace serves one stream at a time.  Calls can be captured into a
 * CUDA graph; give each graph that may run beside another its own handle.
 */
#ifndef GLU_SM103_H_
#define GLU_SM103_H_

#include <stdint.h>

#include "gemm_sm103.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t activation;    /* gemm_activation_t, of the gate */
    const void* bias;      /* device, 2F elements (gate, up), or NULL */
    int32_t bias_dtype;    /* GEMM_F16, GEMM_BF16 or GEMM_F32 */
    void* P;               /* device, M x 2F of H's type, or NULL: not stored */
    int64_t ldp;           /* >= 2F */
} glu_forward_t;

/*
 * glu_forward: H = act(X Wg^T + bg) * (X Wu^T + bu).
 *   dt.a = dt.b: type of X and W; dt.c: type of H and P.
 * M == 0 or F == 0 is a no-op; K == 0 gives P = bias (or 0) without reading X
 * or W.  Returns INVALID_VALUE for opt == NULL, a bad argument, an unknown
 * activation or bias type; otherwise as gemm_run.
 */
gemm_status_t glu_forward(gemm_handle_t h, int64_t M, int64_t F, int64_t K,
                          const void* X, int64_t ldx, const void* W, int64_t ldw,
                          void* H, int64_t ldh, gemm_dtypes_t dt, const glu_forward_t* opt,
                          gemm_stream_t stream);

/* The plan glu_forward would use (host logic only; as gemm_plan_query).  The
 * plan's N is 2F: block_n counts gate and up columns together, and a swapped
 * plan's block_m gate and up rows together. */
gemm_status_t glu_plan_query(int64_t M, int64_t F, int64_t K, const void* X, int64_t ldx,
                             const void* W, int64_t ldw, const void* H, int64_t ldh,
                             gemm_dtypes_t dt, const glu_forward_t* opt, int32_t num_sms,
                             int32_t smem_optin, gemm_plan_t* out);

typedef struct {
    int32_t activation;    /* gemm_activation_t, as in the forward pass */
    int32_t p_dtype;       /* type of P (F16, BF16 or F32) */
    void* dP;              /* M x 2F of dH's type, required; may be P itself (same
                              type and leading dimension) */
    int64_t lddp;
    void* dX;              /* M x K, or NULL: not computed */
    int64_t lddx;
    int32_t dx_dtype;
    void* dW;              /* 2F x K, or NULL: not computed */
    int64_t lddw;
    int32_t dw_dtype;
    float beta_w;          /* 0: dW is overwritten and not read; 1: accumulated */
    void* dbias;           /* 2F elements, or NULL: not computed */
    int32_t dbias_dtype;
} glu_backward_t;

/*
 * glu_backward: dP, and dX, dW, dbias where asked for.
 *   dtype: the type of dH, X, W and dP.  X may be NULL when dW is, W when dX is.
 * M == 0 leaves dW = beta_w * dW and dbias = 0.  Returns as glu_forward.
 */
gemm_status_t glu_backward(gemm_handle_t h, int64_t M, int64_t F, int64_t K,
                           const void* dH, int64_t lddh, const void* P, int64_t ldp,
                           const void* X, int64_t ldx, const void* W, int64_t ldw,
                           int32_t dtype, const glu_backward_t* opt, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GLU_SM103_H_ */
