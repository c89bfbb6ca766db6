/*
 * gemmq_i8.h -- the int8 half of libgemmq's C ABI: a linear layer on int8
 * weights with one scale per output channel and int8 activations with one scale
 * per token, its gradient with respect to the activations, and the softmax
 * cross-entropy over a vocabulary that reads such weights (a language-model
 * head) without keeping the logits, with its gradient; and what a decoder has
 * between such products.  gemmq.h holds the K-quant half, the status codes and
 * gemmq_status_str.
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
 *  - No output may overlap an input, another output or the workspace, but where an
 *    entry says that it may be an input itself.
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

#define GEMMQ_I8_ABI_VERSION 2

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
 * Y may lie in X's place: X is quantized before anything of Y is written.
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

/* ---------------------------------------------------------------------------
 * What stands between the int8 products of a decoder.
 * ------------------------------------------------------------------------- */

/*
 * Residual addition, root-mean-square norm and quantization, of each row:
 *   h = x + r                      rounded to the rows' type (r == NULL: h = x)
 *   p[k] = h[k] * w[k]             in f32
 *   Q, s0 = gemmq_quantize_i8 of p
 *   s = s0 * rstd,  rstd = 1 / sqrt(mean_k h[k]^2 + eps)
 * so that s[m] * Q[m, k] is the quantized norm(h) * w: rstd is one positive factor
 * of a row, which cancels in p / max|p|, and the integers do not depend on it.  The sum
 * of squares is in 64 bits; s is rounded once.
 * A row whose p is not all finite has s = NaN and Q = 0, as in gemmq_quantize_i8.
 *   type      of X, R and H.   R  [M, K] or NULL.
 *   H, ldh    [M, K] or NULL: receives h, and may be X or R itself (the same
 *             pointer and pitch; otherwise it overlaps neither).
 *   w         f32 [K].   eps  >= 0 and finite.
 *   Q, ldq, s as in gemmq_quantize_i8.
 * Errors: as gemmq_quantize_i8, and GEMMQ_E_INVALID_ARG for eps.
 */
int gemmq_rms_i8(int type, const void *X, int64_t ldx, const void *R, int64_t ldr, void *H,
                 int64_t ldh, const float *w, float eps, int8_t *Q, int64_t ldq, float *s,
                 int64_t M, int64_t K, void *stream);

/* Workspace bytes of gemmq_rms_i8_grad with a dw (without one none is needed).  Here and for
   the two entries below 0 is also the size for arguments that the entry refuses, and where it
   needs no workspace: ws may be NULL then. */
size_t gemmq_rms_i8_grad_workspace(int type, int64_t M, int64_t K);

/*
 * The gradient of norm(h) * w (the quantizer's rounding taken as the identity), with
 * n = h * rstd and d = dy * w:
 *   dX[m, k] = rstd (d[k] - n[k] mean_j d[j] n[j])  (+ dH[m, k])
 *   dw[k]    = sum_m dY[m, k] n[m, k]
 * dX is the gradient with respect to x and to r, where dH is what arrives at h by the
 * residual path.
 *   type  of H, dY, dH and dX, all [M, K].   dH  may be NULL.
 *   dX    may be H, dY or dH itself (the same pointer and pitch).
 *   dw    f32 [K], overwritten (zeros where M == 0), or NULL: not computed.
 *   ws    may be NULL where dw is.
 * A row of zeros has rstd = 0 where eps is 0, as it has s = 0 in gemmq_rms_i8: dX is dH, or 0,
 * and dw has nothing of it.
 * Errors: as gemmq_rms_i8, and GEMMQ_E_INVALID_ARG for a workspace that is too small.
 */
int gemmq_rms_i8_grad(int type, const void *H, int64_t ldh, const float *w, float eps,
                      const void *dY, int64_t lddy, const void *dH, int64_t lddh, void *dX,
                      int64_t lddx, float *dw, int64_t M, int64_t K, void *ws, size_t ws_bytes,
                      void *stream);

/* The activations, act(z); at an infinite z act and act' are their limits. */
#define GEMMQ_ACT_NONE 0
#define GEMMQ_ACT_SILU 1      /* z / (1 + exp(-z)) */
#define GEMMQ_ACT_GELU 2      /* z (1 + erf(z / sqrt 2)) / 2 */
#define GEMMQ_ACT_GELU_TANH 3 /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
#define GEMMQ_ACT_RELU 4      /* max(z, 0) */

/*
 * gemmq_gemm_i8 with an activation and a residual in its epilogue:
 *   z[m, n] = sx[m] * sw[n] * sum_k Xq[m, k] * W[n, k]  (+ bias[n])
 *   Y[m, n] = act(z[m, n])  (+ R[m, n])
 * in f32, rounded once to Y's type.
 *   R, ldr  [M, N] of Y's type, or NULL; Y may be R itself (the same pointer and pitch).
 *   Z, ldz  [M, N] of Y's type, or NULL: receives z, rounded, for gemmq_act_grad; not R.
 * Errors: as gemmq_gemm_i8, and GEMMQ_E_INVALID_ARG for an unknown act, or one matrix as
 *         two of the results.
 */
int gemmq_gemm_i8_act(const int8_t *W, int64_t ldw, const float *sw, const int8_t *Xq, int64_t ldq,
                      const float *sx, const float *bias, int act, const void *R, int64_t ldr,
                      int ytype, void *Y, int64_t ldy, void *Z, int64_t ldz, int64_t M, int64_t N,
                      int64_t K, void *stream);

/* Quantize X into Xq and sx, then gemmq_gemm_i8_act: the same bits as the two calls, also
   where Y or Z lies in X's place. */
int gemmq_linear_i8_act(const int8_t *W, int64_t ldw, const float *sw, int xtype, const void *X,
                        int64_t ldx, int8_t *Xq, int64_t ldq, float *sx, const float *bias,
                        int act, const void *R, int64_t ldr, int ytype, void *Y, int64_t ldy,
                        void *Z, int64_t ldz, int64_t M, int64_t N, int64_t K, void *stream);

/*
 * A gated pair of matrices on the same activations, both [N, K]:
 *   z[m, n] = sx[m] * sw[n] * sum_k Xq[m, k] * W[n, k]  (+ bias[n])
 *   u[m, n] = sx[m] * swu[n] * sum_k Xq[m, k] * Wu[n, k]  (+ biasu[n])
 *   Y[m, n] = act(z[m, n]) * u[m, n]
 * in f32, rounded once to Y's type.
 *   Z, ldz and U, ldu  [M, N] of Y's type, or NULL: receive z and u, rounded.
 * M * 2 N counts against GEMMQ_I8_MAX_OUTPUTS.
 * Errors: as gemmq_gemm_i8_act.
 */
int gemmq_gemm_i8_gate(const int8_t *W, int64_t ldw, const float *sw, const int8_t *Wu,
                       int64_t ldwu, const float *swu, const int8_t *Xq, int64_t ldq,
                       const float *sx, const float *bias, const float *biasu, int act, int ytype,
                       void *Y, int64_t ldy, void *Z, int64_t ldz, void *U, int64_t ldu, int64_t M,
                       int64_t N, int64_t K, void *stream);

/* Quantize X into Xq and sx, then gemmq_gemm_i8_gate: the same bits as the two calls, also
   where Y, Z or U lies in X's place. */
int gemmq_linear_i8_gate(const int8_t *W, int64_t ldw, const float *sw, const int8_t *Wu,
                         int64_t ldwu, const float *swu, int xtype, const void *X, int64_t ldx,
                         int8_t *Xq, int64_t ldq, float *sx, const float *bias, const float *biasu,
                         int act, int ytype, void *Y, int64_t ldy, void *Z, int64_t ldz, void *U,
                         int64_t ldu, int64_t M, int64_t N, int64_t K, void *stream);

/* Workspace bytes of gemmq_act_grad with a db or dbu (without them none is needed). */
size_t gemmq_act_grad_workspace(int type, int64_t M, int64_t N);

/*
 * The gradients behind the two products above, which gemmq_linear_i8_grad takes on to
 * the activations:
 *   without U:  dZ = dY act'(Z)
 *   with U:     dZ = dY U act'(Z),  dU = dY act(Z)
 *   db[n] = sum_m dZ[m, n],  dbu[n] = sum_m dU[m, n]   of the values before their rounding
 * (relu' (0) = 0; the residual's gradient is dY itself).
 *   type  of Z, U, dY, dZ and dU, all [M, N].   U and dU  both or neither (NULL).
 *   dZ    may be Z or dY itself, dU may be U or dY itself, not both dY (the same
 *         pointer and pitch).
 *   db, dbu  f32 [N], overwritten (zeros where M == 0), or NULL: not computed; dbu
 *         only with U.
 *   ws    may be NULL where db and dbu are.
 * Errors: as gemmq_quantize_i8, and GEMMQ_E_INVALID_ARG for an unknown act, one of U
 *         and dU alone, a dbu without U, db and dbu the same vector, or a workspace that
 *         is too small.
 */
int gemmq_act_grad(int act, int type, const void *Z, int64_t ldz, const void *U, int64_t ldu,
                   const void *dY, int64_t lddy, void *dZ, int64_t lddz, void *dU, int64_t lddu,
                   float *db, float *dbu, int64_t M, int64_t N, void *ws, size_t ws_bytes,
                   void *stream);

/* Workspace bytes of gemmq_sample. */
size_t gemmq_sample_workspace(int64_t M, int64_t N);

/*
 * One token a row from its logits, with the row's own settings and random number.
 * The tokens of a row stand in the order of their logits, the largest first, equal
 * ones (+0 and -0 are equal) by their index, with the weights
 *   e = exp((z - max z) / temperature)
 * and the first of them are kept: no more than
 *   top_k  of them (<= 0: no limit);
 *   top_p  < 1: the fewest whose weights' sum is at least top_p times that of all
 *          that top_k leaves (<= 0: one; >= 1 or NaN: no limit);
 *   min_p  > 0: those with e >= min_p (above 1 as 1; NaN: no limit);
 * one at least.  Of these the token is the first where the running sum of the weights
 * is more than u times their whole sum.
 * temperature <= 0: the largest logit, whatever the rest says.
 *   Z, ldz       [M, N], N >= 1 (GEMMQ_E_SHAPE otherwise).  -inf takes a token out.
 *   temperature, top_p, min_p  f32 [M], top_k  int32 [M]; each may be NULL: 1, and no
 *                limits.
 *   u            f32 [M], in [0, 1) (below 0 or NaN as 0, from 1 on as the largest f32
 *                below 1).
 *   token        int64 [M].   logprob  f32 [M] or NULL: the logarithm of the token's
 *                share of the kept tokens' weights.
 * A row without a token to draw (a NaN, a +inf, nothing but -inf, or a temperature
 * that is NaN or +inf) has token -1 and logprob NaN.
 * Weights are fixed-point numbers with 62 - ceil(log2 N) bits (50 at most) behind the
 * point, the largest one 1, and their sums are exact: a result does not depend on the order
 * of anything.  A weight below half a unit is zero, and drawn by no u.
 * Errors: as gemmq_loss_i8.
 */
int gemmq_sample(int type, const void *Z, int64_t ldz, const float *temperature,
                 const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                 int64_t *token, float *logprob, int64_t M, int64_t N, void *ws, size_t ws_bytes,
                 void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMMQ_I8_H */
