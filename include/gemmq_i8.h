/*
 * gemmq_i8.h -- the int8 half of libgemmq's C ABI: a linear layer on int8
 * weights with one scale per output channel and int8 activations with one scale
 * per token, its gradient with respect to the activations, and the softmax
 * cross-entropy over a vocabulary that reads such weights (a language-model
 * head) without keeping the logits, with its gradient.  gemmq.h holds the
 * K-quant half, the status codes and gemmq_status_str.
 *
 * The values:  w[n, k] = sw[n] * W[n, k],   x[m, k] = sx[m] * Xq[m, k].
 *
 * Conventions (those of gemmq.h where not said otherwise):
 *  - Pointers are DEVICE pointers on the current HIP device; `stream` is a
 *    hipStream_t as void* (NULL: the default stream).  GEMMQ_OK means the work
 *    is enqueued on that stream.  The library allocates nothing, keeps no state
 *    between calls, never synchronises, and enqueues kernels only, so every call
 *    may be captured into a graph.  A negative status means nothing was launched.
 *  - Matrices are row-major with a row pitch: W is int8 [N, K] with row n at
 *    W + n*ldw bytes, Xq int8 [M, K] with row m at Xq + m*ldq; both pitches are
 *    multiples of 16 bytes, at least K and at most GEMMQ_I8_MAX_PITCH, and both
 *    bases 16-byte aligned.  The bytes of a row from K to the next multiple of 16
 *    are read (the last row's too) but never enter a result, whatever they hold,
 *    and are never written; a row's bytes beyond those are not touched.
 *    X, Y, dY and dX have their pitch in elements, at least their width, and any
 *    alignment of their element type; wider accesses are used where base and
 *    pitch allow them.
 *  - Element types: GEMMQ_F32, GEMMQ_BF16, GEMMQ_F16.
 *  - 1 <= K <= GEMMQ_I8_MAX_K: the int32 sums cannot overflow, also with -128 in
 *    both matrices.  M and N up to GEMMQ_I8_MAX_ROWS.  One launch holds all output
 *    tiles: M * N of a product or a loss and M * K of a gradient fit up to
 *    GEMMQ_I8_MAX_OUTPUTS, whatever the shape; beyond it a call may be refused with
 *    GEMMQ_E_SHAPE.  M == 0 is a valid empty call: nothing is touched.
 *  - `ws` is scratch memory of at least the bytes that the entry's ..._workspace
 *    function gives for the same arguments, 16-byte aligned; its contents before
 *    the call do not matter and are not defined after it.  Calls that can run at
 *    the same time (other streams, graphs replayed together) need workspaces of
 *    their own, as they need outputs of their own.
 *  - No output may overlap an input, another output or the workspace.
 *  - Results do not depend on timing: no floating-point atomics, every sum has a
 *    fixed order for given arguments.  A row m of a result depends on row m of the
 *    activations only, so a row with a NaN does not touch the others.
 */
#ifndef GEMMQ_I8_H
#define GEMMQ_I8_H

#include <stddef.h>
#include <stdint.h>

#include "gemmq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMMQ_I8_ABI_VERSION 1

#define GEMMQ_F32 0
#define GEMMQ_BF16 1
#define GEMMQ_F16 2

#define GEMMQ_I8_MAX_K 131071        /* 2^14 * 131071 < 2^31 */
#define GEMMQ_I8_MAX_ROWS 16777216   /* 2^24 rows of any matrix */
#define GEMMQ_I8_MAX_PITCH 1048576   /* bytes between rows of an int8 matrix */
#define GEMMQ_I8_MAX_OUTPUTS 68719476736 /* 2^36: outputs that always fit a launch */

/* GEMMQ_I8_ABI_VERSION of the library that was loaded.  Never fails. */
int gemmq_i8_abi_version(void);

/*
 * Quantize rows to int8 with one f32 scale each -- activations per token, or
 * weights per output channel:
 *   s[m] = max_k |x[m, k]| / 127                    (f32, correctly rounded)
 *   q[m, k] = round-half-even(x[m, k] / s[m])       (f32, correctly rounded
 *             division), clamped to [-127, 127]
 * A row whose s is 0 (all zeros, or too small for an f32 scale) has q = 0; a row
 * with an infinity or a NaN has s = NaN and q = 0, so that whatever is computed
 * from that row is NaN.
 *   xtype, X, ldx  the rows, [M, K].
 *   Q, ldq         int8 [M, K]; the K values of each row are written.
 *   s              f32 [M], 4-byte aligned.
 * Errors: GEMMQ_E_INVALID_ARG (null pointer with M > 0, M < 0, unknown type),
 *         GEMMQ_E_SHAPE (K, M or a pitch outside the limits above),
 *         GEMMQ_E_ALIGNMENT, GEMMQ_E_DEVICE, GEMMQ_E_LAUNCH.
 */
int gemmq_quantize_i8(int xtype, const void *X, int64_t ldx, int8_t *Q, int64_t ldq, float *s,
                      int64_t M, int64_t K, void *stream);

/*
 * Y[m, n] = sx[m] * sw[n] * sum_k Xq[m, k] * W[n, k]  (+ bias[n])
 * The sum is exact in int32; the scaling is in f32, rounded once to Y's type.
 *   sw    f32 [N]; bias  f32 [N] or NULL; sx  f32 [M].
 *   ytype, Y, ldy  [M, N], overwritten (the N values of each row).
 * N == 0 is a valid empty call.
 * Errors: as gemmq_quantize_i8.
 */
int gemmq_gemm_i8(const int8_t *W, int64_t ldw, const float *sw, const int8_t *Xq, int64_t ldq,
                  const float *sx, const float *bias, int ytype, void *Y, int64_t ldy, int64_t M,
                  int64_t N, int64_t K, void *stream);

/*
 * The whole linear layer: quantize X into Xq and sx, then gemmq_gemm_i8 -- the
 * same bits as the two calls, for Xq, sx and Y.  N == 0 still quantizes.
 * Errors: those of the two calls; nothing is launched on an error.
 */
int gemmq_linear_i8(const int8_t *W, int64_t ldw, const float *sw, int xtype, const void *X,
                    int64_t ldx, int8_t *Xq, int64_t ldq, float *sx, const float *bias, int ytype,
                    void *Y, int64_t ldy, int64_t M, int64_t N, int64_t K, void *stream);

/* Workspace bytes of gemmq_linear_i8_grad (0 for arguments it refuses). */
size_t gemmq_linear_i8_grad_workspace(int type, int64_t M, int64_t N, int64_t K);

/*
 * The gradient of the linear layer with respect to its activations:
 *   dX[m, k] = sum_n dY[m, n] * sw[n] * W[n, k]
 * (the rounding of the quantizer is taken as the identity, as is usual: dX is
 * the gradient with respect to the dequantized x).  The products run on the
 * matrix cores with the weights exact in bf16 and dY * sw, an f32 product,
 * written as a sum of bf16 numbers: one for GEMMQ_BF16 (8 bits, the precision
 * of dY itself; two up to M == 8), two for GEMMQ_F16 (16 bits), three for
 * GEMMQ_F32 (24 bits, all of an f32); the sums are f32.  For 9 to 128 rows of
 * GEMMQ_BF16 with N a multiple of 8 and rows on 16 bytes, dY enters as it is and
 * sw * W is rounded to bf16 instead: the same number of roundings, another of the
 * two factors.
 *   type   of dY and dX.   dY, lddy  [M, N].   dX, lddx  [M, K], overwritten.
 * N == 0 writes zeros.
 * Errors: as gemmq_quantize_i8, and GEMMQ_E_INVALID_ARG for a workspace that is
 *         NULL or smaller than gemmq_linear_i8_grad_workspace says.
 */
int gemmq_linear_i8_grad(const int8_t *W, int64_t ldw, const float *sw, int type, const void *dY,
                         int64_t lddy, void *dX, int64_t lddx, int64_t M, int64_t N, int64_t K,
                         void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes of gemmq_loss_i8 (0 for arguments it refuses). */
size_t gemmq_loss_i8_workspace(int64_t M, int64_t N, int64_t K);

/*
 * Softmax cross-entropy over a vocabulary of N rows, with the logits
 * z[m, n] = sx[m] * sw[n] * sum_k Xq[m, k] * W[n, k] never written to memory:
 *   lse[m]  = log sum_n exp(z[m, n])
 *   loss[m] = lse[m] - z[m, target[m]]
 * target[m] < 0 (an ignored position): loss[m] = 0, lse[m] as always, to a rounding.
 * target[m] >= N: loss[m] = NaN.  N >= 1 (GEMMQ_E_SHAPE otherwise).
 *   target  int64 [M], 8-byte aligned.   loss, lse  f32 [M], overwritten.
 * Errors: as gemmq_linear_i8_grad.
 */
int gemmq_loss_i8(const int8_t *W, int64_t ldw, const float *sw, const int8_t *Xq, int64_t ldq,
                  const float *sx, const int64_t *target, float *loss, float *lse, int64_t M,
                  int64_t N, int64_t K, void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes of gemmq_loss_i8_grad (0 for arguments it refuses). */
size_t gemmq_loss_i8_grad_workspace(int type, int64_t M, int64_t N, int64_t K);

/*
 * The gradient of sum_m dloss[m] * loss[m] with respect to the dequantized
 * hidden states, the logits computed once more from Xq a piece of the
 * vocabulary at a time:
 *   dX[m, k] = dloss[m] * sum_n (exp(z[m, n] - lse[m]) - [n == target[m]]) * sw[n] * W[n, k]
 * Rows with target[m] < 0 are zero (whatever dloss and lse hold); with
 * target[m] >= N NaN.
 *   lse    f32 [M], from gemmq_loss_i8 on the same arguments.
 *   dloss  f32 [M].   type, dX, lddx  [M, K], overwritten.
 * `type` also sets the precision of the softmax factor: one bf16 number for
 * GEMMQ_BF16 (two up to M == 8, and the target's to 16 bits for any M), two for
 * GEMMQ_F16, three for GEMMQ_F32.
 * Errors: as gemmq_loss_i8.
 */
int gemmq_loss_i8_grad(const int8_t *W, int64_t ldw, const float *sw, const int8_t *Xq,
                       int64_t ldq, const float *sx, const int64_t *target, const float *lse,
                       const float *dloss, int type, void *dX, int64_t lddx, int64_t M, int64_t N,
                       int64_t K, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMMQ_I8_H */
