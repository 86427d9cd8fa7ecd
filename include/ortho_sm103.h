/*
 * ortho_sm103.h -- C ABI of the GB300 (sm_103a) orthogonalised update: a weight
 * matrix's update (its momentum) brought near the closest matrix with orthonormal
 * rows or columns by Newton-Schulz steps, as the Muon optimiser does, for one
 * matrix or a batch of them.
 *
 *     X = G / (||G||_F + eps)                       (transposed where rows > cols)
 *     steps times:  A = X X^T,  X = a X + (b A + c A^2) X
 *     O = round(scale * X)                          (transposed back)
 *
 * with (a, b, c) of each step from the caller; (3.4445, -4.7750, 2.0315) five times
 * is the optimiser's usual choice.
 *
 * Precision.  The products are the tensor core's: FP16 operands, FP32 sums.  A and
 * b A + c A^2 are rounded to FP16 but for their diagonals, which are kept in FP32.
 * X is carried as FP16 and a remainder of a byte (2^-20 of X together), of two bytes
 * (2^-28) before steps that with those behind them enlarge a rounding by more than 512
 * (the product of their a); the products take the FP16 part.
 * Besides its own rounding to BF16 (0.0017 of its norm) O is off by
 *   five usual steps: 0.0002 to 0.0016 of its norm, on spectra from rank 1 to noise (the
 *     most where rank 1 to 4 meets sides of thousands, and of noise on sides of tens; a
 *     handful of elements can be off by 0.006);
 *   eight: 0.001 to 0.002 where no singular value is far below 10^-6 of the largest.
 * An error in the directions of singular values near 0 grows by a (3.4) in every step,
 * and the sums' FP32 errors, sqrt(sides) 2^-25, are one: of rank 1 to 4 O is off by 0.002
 * (256 x 1024) to 0.018 (2048 x 2047) after eight steps and by ten times that after ten,
 * as it is in FP32 arithmetic throughout.  Values of X, A and
 * b A + c A^2 up to 32 in magnitude are held: coefficients that keep the singular
 * values near 1 stay far below.
 * A and A^2 are symmetric: half their tiles are computed, the others mirrored.
 * The sum of squares is FP32 over up to 32 elements and FP64 from there on, in a fixed
 * order: the same call gives the same bits.
 *
 * A matrix of zeros gives zeros (with eps > 0); one with an infinity or NaN gives
 * NaN everywhere.
 *
 * Layout: row-major, leading dimensions and batch strides in elements, any
 * alignment to the element size.  G is F16, BF16 or F32, O is BF16 and may overlap G
 * or be G: all of G has been read before any of O is written (O holds a part of X
 * between the steps).  Padding is never touched.
 *
 * Ownership, threading, workspace and errors: as gemm_run (gemm_sm103.h), on the
 * handle's device, which has to be current (INVALID_VALUE otherwise): the handle's
 * workspace (ortho_workspace bytes of it) serves one stream at a time.  Calls can be
 * captured into a CUDA graph; give each graph that may run beside another its own
 * handle.
 */
#ifndef ORTHO_SM103_H_
#define ORTHO_SM103_H_

#include <stdint.h>

#include "gemm_sm103.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ORTHO_MAX_STEPS 32
#define ORTHO_MAX_SIDE 65536

typedef struct {
    int32_t steps;               /* 1 .. ORTHO_MAX_STEPS */
    const float* coefficients;   /* HOST, 3 per step (a, b, c), read during the call; finite */
    float eps;                   /* >= 0 and finite */
    float scale;                 /* finite */
} ortho_update_t;

/*
 * ortho_update: O = the orthogonalised G, for each of `batch` matrices.
 *   Matrix i starts at G + i * stride_g and O + i * stride_o; the strides of a batch
 *   above 1 are at least (rows - 1) * ld + cols, ldg and ldo at least cols.
 * batch, rows or cols 0 is a no-op.  Returns INVALID_VALUE for opt == NULL or a bad
 * argument (a side above ORTHO_MAX_SIDE, batch above 65535); otherwise as gemm_run.
 */
gemm_status_t ortho_update(gemm_handle_t h, int64_t batch, int64_t rows, int64_t cols,
                           const void* G, int64_t ldg, int64_t stride_g, int32_t g_dtype,
                           void* O, int64_t ldo, int64_t stride_o, const ortho_update_t* opt,
                           gemm_stream_t stream);

/* Bytes of the handle's workspace that such a call takes; -1 for bad arguments. */
int64_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols);

#ifdef __cplusplus
}
#endif

#endif /* ORTHO_SM103_H_ */
