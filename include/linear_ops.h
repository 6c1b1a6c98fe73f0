/*
 * linear_ops.h -- C ABI of the training and serving operators around a fused
 * product, in libgemm_epi.so (AMD Instinct MI355X, gfx950).
 *
 * ge_linear                  Z = X W^T + bias, D = act(Z) + residual
 * ge_linear_backward         dZ = dD act'(Z); dX = dZ W, dW = dZ^T X, dbias = sum of dZ over rows
 * ge_linear_xent             softmax cross entropy of the logits X W^T, which are never stored
 * ge_linear_xent_backward    its gradients, in pieces of the vocabulary
 * ge_norm_residual           H' = H + scale gate norm_post(Y), X = norm_pre(H')
 * ge_norm_residual_backward  its gradients
 *
 * Every call takes one argument structure (all fields 8 bytes wide), runs its
 * checks on the host before any HIP call, queues kernels on args->stream and
 * returns a gemm_epi_status.  It allocates nothing, synchronises nothing and
 * queues nothing but kernels, so it records into a HIP graph.  Scratch memory
 * comes from the caller: the matching ge_*_workspace call (host only) checks the
 * same arguments, workspace and stream aside, and stores the bytes the call
 * needs; the workspace need not be initialised, is 16-byte aligned, and may be
 * reused once the call's work has completed.
 *
 * Matrices are row-major with unit element stride and a row stride (ld*) in
 * elements, at least the row length; rows start at any element-aligned
 * address.  dtype is GEMM_EPI_F16 or GEMM_EPI_BF16.  All sums, softmax
 * statistics and norms are fp32; each output is rounded once, to nearest-even.
 * Results do not depend on the launch order of anything: no atomics.
 */
#ifndef LINEAR_OPS_H
#define LINEAR_OPS_H

#include <stdint.h>

#include "gemm_epi.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GE_ACT_IDENTITY = 0, GE_ACT_RELU = 1, GE_ACT_GELU = 2, GE_ACT_SILU = 3 } ge_act;
typedef enum { GE_NORM_NONE = 0, GE_NORM_RMS = 1, GE_NORM_LAYER = 2 } ge_norm;

/* Row strides and row lengths (N, K) are at most GE_MAX_COLS, M, T and V at most
 * 2^31 - 257 (2^31 - 1 rows in the norms); hidden is at most GE_MAX_HIDDEN, and
 * GE_MAX_HIDDEN_GRAD in the gradient.  A product of more than 16 rows has fewer
 * than 2^24 tiles of 256 x 256; one past that is refused with the shape status. */
#define GE_MAX_COLS 2097000
#define GE_MAX_HIDDEN 16384
#define GE_MAX_HIDDEN_GRAD 8192

/* X (M, K), W (N, K), bias (N) or NULL, residual (M, N) or NULL, D (M, N), Z
 * (M, N) or NULL (not kept).  act: ge_act; gelu is the exact (erf) form.  D may
 * be the residual itself.  M may be 0. */
typedef struct {
    int64_t M, N, K;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    const void *bias;
    const void *residual;
    int64_t ldr;
    void *D;
    int64_t ldd;
    void *Z;
    int64_t ldz;
    int64_t act, dtype;
    void *workspace;
    int64_t workspace_bytes;
    void *stream;
} ge_linear_args;

/* dD (M, N), X (M, K), W (N, K), Z (M, N) as ge_linear kept it (not read, and
 * may be NULL, for the identity; relu masks: dD where Z <= 0 does not count,
 * whatever it is); dX (M, K), dW (N, K), dbias (N) fp32, each NULL where it is
 * not wanted.  dZ is rounded to the element type as an operand of the two
 * products (dbias sums it unrounded); it is not scaled, so in fp16 it has the
 * range that dD has, less a factor of 1.13 (the largest |act'|): the caller's
 * loss scale keeps both.  With M = 0, dW and dbias are set to zero, and all three
 * may be NULL (an empty dX has no address). */
typedef struct {
    int64_t M, N, K;
    const void *dD;
    int64_t lddd;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    const void *Z;
    int64_t ldz;
    void *dX;
    int64_t lddx;
    void *dW;
    int64_t lddw;
    float *dbias;
    int64_t act, dtype;
    void *workspace;
    int64_t workspace_bytes;
    void *stream;
} ge_linear_backward_args;

/* X (T, K), W (V, K), target (T) int64; loss (T), lse (T) fp32.
 * lse[t] = log sum_v exp(X W^T)[t][v]; loss[t] = lse[t] - (X W^T)[t][target[t]],
 * 0 where target[t] is ignore_index, NaN where it is neither that nor in
 * [0, V).  T may be 0. */
typedef struct {
    int64_t T, V, K;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    const int64_t *target;
    int64_t ignore_index;
    float *loss;
    float *lse;
    int64_t dtype;
    void *workspace;
    int64_t workspace_bytes;
    void *stream;
} ge_linear_xent_args;

/* dloss (T) fp32, lse (T) from ge_linear_xent; dX (T, K), dW (V, K), each NULL
 * where it is not wanted.  P = (exp(logit - lse) - [v == target]) dloss, zero in
 * ignored rows, is formed one piece of the vocabulary at a time and rounded to
 * the element type as an operand (fp16: after a common factor for all rows, so that
 * an entry is off by its rounding and at most 2^-39 of the largest |dloss|).  A
 * row whose target is out of range makes its gradients NaN.  A piece of P is
 * 128 MiB, or 8192 columns where that is more: past 8192 rows the workspace
 * grows by 16 KiB a row, and 4 K bytes for dX between the pieces.  With T = 0, dW is set to zero, and both may be NULL. */
typedef struct {
    int64_t T, V, K;
    const float *dloss;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    const int64_t *target;
    const float *lse;
    int64_t ignore_index;
    void *dX;
    int64_t lddx;
    void *dW;
    int64_t lddw;
    int64_t dtype;
    void *workspace;
    int64_t workspace_bytes;
    void *stream;
} ge_linear_xent_backward_args;

/* H, H_out (T, H) of stream_dtype (the element type or GEMM_EPI_F32), Y, X (T, H)
 * and w_post, w_pre (H), gate (G, H) of dtype; each of w_post, w_pre, gate may
 * be NULL (ones; G is then 1).  Gate row g serves rows g T/G .. (g+1) T/G - 1.
 * H' = H + scale gate norm_post(Y) w_post, X = norm_pre(H') w_pre from the
 * unrounded H'.  RMS: v / sqrt(mean v^2 + eps); LAYER: (v - mean) /
 * sqrt(var + eps); NONE (post only): v, and w_post is not read.  H_out may be
 * H.  T may be 0. */
typedef struct {
    int64_t T, hidden, G;
    const void *H;
    int64_t ldh;
    const void *Y;
    int64_t ldy;
    const void *w_post;
    const void *w_pre;
    const void *gate;
    int64_t post, pre;
    double scale, eps;
    void *H_out;
    int64_t ldho;
    void *X;
    int64_t ldx;
    int64_t dtype, stream_dtype;
    void *stream;
} ge_norm_residual_args;

/* dX (T, H) of dtype, dH_out (T, H) and H_out (T, H) of stream_dtype, Y (T, H);
 * dH of stream_dtype, dY of dtype, dw_post, dw_pre (H) and dgate (G, H) fp32,
 * each of the last three NULL where it is not wanted.  With T = 0 the last
 * three are set to zero. */
typedef struct {
    int64_t T, hidden, G;
    const void *dX;
    int64_t lddx;
    const void *dH_out;
    int64_t lddho;
    const void *H_out;
    int64_t ldho;
    const void *Y;
    int64_t ldy;
    const void *w_post;
    const void *w_pre;
    const void *gate;
    int64_t post, pre;
    double scale, eps;
    void *dH;
    int64_t lddh;
    void *dY;
    int64_t lddy;
    float *dw_post;
    float *dw_pre;
    float *dgate;
    int64_t dtype, stream_dtype;
    void *workspace;
    int64_t workspace_bytes;
    void *stream;
} ge_norm_residual_backward_args;

int ge_linear(const ge_linear_args *args);
int ge_linear_workspace(const ge_linear_args *args, int64_t *bytes);
int ge_linear_backward(const ge_linear_backward_args *args);
int ge_linear_backward_workspace(const ge_linear_backward_args *args, int64_t *bytes);
int ge_linear_xent(const ge_linear_xent_args *args);
int ge_linear_xent_workspace(const ge_linear_xent_args *args, int64_t *bytes);
int ge_linear_xent_backward(const ge_linear_xent_backward_args *args);
int ge_linear_xent_backward_workspace(const ge_linear_xent_backward_args *args, int64_t *bytes);
int ge_norm_residual(const ge_norm_residual_args *args);
int ge_norm_residual_backward(const ge_norm_residual_backward_args *args);
int ge_norm_residual_backward_workspace(const ge_norm_residual_backward_args *args, int64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_OPS_H */
