/*
 * w8a8_block.h -- the operators beside the 8-bit linear in a transformer
 * block: low-rank adapters of many requests added to a shared projection,
 * layer norm, both with their backward passes, and layer norm fused with the
 * row-wise activation quantizer.
 *
 * Ownership, execution and errors are those of w8a8.h: device pointers owned
 * by the caller, arguments checked on the host before anything is launched,
 * kernels enqueued on `stream` without allocation, clearing or
 * synchronization (graph-capturable), sizes of 0 a successful no-op (but sums
 * over no rows are written as zero), base pointers 16-byte aligned.  An output
 * overlaps no other argument, except where a declaration says that it may be
 * one of them.  Results do not depend on the order in which
 * workgroups run (no atomics): the same call gives the same bits.  Infinities
 * and NaN follow the formulas and stay in the rows, requests and columns
 * whose formulas hold them.
 */
#ifndef W8A8_BLOCK_H_
#define W8A8_BLOCK_H_

#include "w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    W8A8_BF16 = 0, /* bfloat16 bit patterns */
    W8A8_F32 = 1
} w8a8_dtype;

/* ------------------------------------------------------------------ adapters
 *
 * A pool of L low-rank adapters (a [L, R, K], b [L, N, R]: nn.Linear layouts,
 * as svdq_linear's l1 and l2) beside one shared projection.  The rows of X
 * are the tokens of a batch of requests, one request after the other; each
 * request uses one adapter of the pool or none.
 *
 * The plan.  Which rows use which adapter is laid out once per batch, on the
 * host, and serves every projection of every layer that the batch passes:
 * tiles of at most W8A8_LORA_TILE_ROWS rows of one request, as int32
 * {first row, rows, adapter (-1: none), 0}, ordered by adapter and row, then
 * L + 1 int32: adapter l has the tiles first[l] .. first[l + 1] - 1.  The
 * caller copies the 4 T + L + 1 integers to the device.  Entries that do not
 * fit the call's M and L are skipped by the kernels, never followed.
 */
#define W8A8_LORA_TILE_ROWS 64

/*
 * Builds the plan of S requests in host memory: lengths [S] (>= 0, zero
 * allowed), adapters [S] (-1 .. L - 1).  Writes the tile count T to *tiles
 * and, if plan is not NULL, the 4 T + L + 1 integers to plan (capacity
 * integers long, else W8A8_ERR_SHAPE).  Call it with plan = NULL for the
 * size.  The sum of the lengths is at most 2^30, T at most 2^24, L is in
 * [1, 65535] (W8A8_ERR_SHAPE); a negative length or an adapter outside the pool is
 * W8A8_ERR_INVALID_ARG.  All pointers are host pointers.
 */
w8a8_status lora_plan(const int64_t *lengths, const int32_t *adapters, int64_t S, int64_t L, int32_t *plan,
                      int64_t capacity, int64_t *tiles);

/*
 * out[m, n] = bf16(base[m, n] + sum_j u[m, j] * b[l, n, j]),
 * u[m, j]   = scale[l] * sum_k x[m, k] * a[l, j, k]   for j < ranks[l], else 0
 * for every row m of a tile with adapter l; rows without an adapter have
 * u = 0 and out = base.  f32 sums; u is multiplied into b as a pair of bf16
 * halves (~16 significant bits; what lies below 2^-133, bf16's smallest step,
 * counts as 0).
 *   x bf16 [M, ldx] (first K columns); a bf16 [L, R, K]; b bf16 [L, N, R];
 *   scale f32 [L] or NULL (1); ranks int32 [L] or NULL (R), clamped to
 *   [0, R]: entries of a and b beyond an adapter's rank are never used,
 *   whatever they hold.  plan: device copy of lora_plan's T tiles.
 *   base bf16 [M, ldbase] or NULL (0); out bf16 [M, ldout], may be base
 *   (in place, same stride).  u f32 [M, R] or NULL: what lora_backward takes.
 *   workspace lora_forward_workspace_bytes(M, R) bytes, used if u is NULL.
 * Rows in no tile are not written.
 * Shape rules: M >= 0, 0 <= T <= 2^24, 1 <= L <= 65535; K, N, R, strides
 * multiples of 8; 8 <= R <= 128 (else W8A8_ERR_INVALID_ARG), 8 <= K, N <= 2^22,
 * M <= 2^30, strides from their width up to 2^22.
 */
size_t lora_forward_workspace_bytes(int64_t M, int64_t R);
w8a8_status lora_forward(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, const uint16_t *a, const uint16_t *b,
                         int64_t L, int64_t N, int64_t R, const float *scale, const int32_t *ranks,
                         const int32_t *plan, int64_t T, const uint16_t *base, int64_t ldbase, uint16_t *out,
                         int64_t ldout, float *u, void *workspace, hipStream_t stream);

/*
 * Gradients of lora_forward for a frozen shared projection, with
 * g[m, j] = scale[l] * sum_n dy[m, n] * b[l, n, j] for j < ranks[l]:
 *   dx[m, k]    = bf16(base[m, k] + sum_j g[m, j] * a[l, j, k])
 *   da[l, j, k] = sum of g[m, j] * x[m, k] over the rows of adapter l
 *   db[l, n, j] = sum of dy[m, n] * u[m, j] over the rows of adapter l
 *   (zero for adapters without rows and for j >= ranks[l]).
 *   dy bf16 [M, lddy]; x, a, b, scale, ranks, plan as in the forward call;
 *   u f32 [M, R] from it.  base bf16 [M, ldbase] or NULL: the shared
 *   projection's own input gradient (w8a8_linear_backward_dx), may be dx.
 *   dx bf16 [M, lddx]; da f32 [L, R, K]; db f32 [L, N, R], f32 accurate (g and
 *   u are three bf16 parts: all 24 bits of values above 2^-110).
 *   dx may be NULL (no input gradient); da and db may both be NULL.
 *   workspace lora_backward_workspace_bytes(M, T, K, N, R, L) bytes.
 * Shape rules as lora_forward.
 */
size_t lora_backward_workspace_bytes(int64_t M, int64_t T, int64_t K, int64_t N, int64_t R, int64_t L);
w8a8_status lora_backward(const uint16_t *dy, int64_t M, int64_t N, int64_t lddy, const uint16_t *x, int64_t K,
                          int64_t ldx, const float *u, const uint16_t *a, const uint16_t *b, int64_t L, int64_t R,
                          const float *scale, const int32_t *ranks, const int32_t *plan, int64_t T,
                          const uint16_t *base, int64_t ldbase, uint16_t *dx, int64_t lddx, float *da, float *db,
                          void *workspace, hipStream_t stream);

/* ---------------------------------------------------------------- layer norm
 *
 * mean[m] = sum_k x[m, k] / K,  rstd[m] = 1 / sqrt(var[m] + eps) with the
 * biased variance about that mean,  h = (x - mean) * rstd,
 * y[m, k] = h[m, k] * weight[k] + bias[k].
 *   x, y of type xt (bf16 or f32), rows of K elements ldx, ldy apart;
 *   weight, bias [K] of type wt, each may be NULL (1, 0); mean, rstd f32 [M],
 *   each may be NULL.  y may be x (same stride).  Statistics and arithmetic
 *   in f32, one rounding to xt.
 * Shape rules: M >= 0, 1 <= K <= 2^24, strides from K up to 2^24 and any
 * alignment of the rows; eps >= 0 and finite (W8A8_ERR_INVALID_ARG).
 */
w8a8_status layer_norm_forward(w8a8_dtype xt, const void *x, int64_t M, int64_t K, int64_t ldx, w8a8_dtype wt,
                               const void *weight, const void *bias, float eps, void *y, int64_t ldy, float *mean,
                               float *rstd, hipStream_t stream);

/*
 * Gradients of layer_norm_forward from its mean and rstd, with
 * t = dy * weight:
 *   dx = rstd * (t - <t> - h * <t * h>), <.> the mean over a row;
 *   dweight[k] = sum_m dy * h,  dbias[k] = sum_m dy   (f32 [K]).
 *   dy, x, dx of type xt, weight of type wt or NULL; dx, dweight, dbias may
 *   each be NULL; dx may be dy (same stride).
 *   workspace layer_norm_backward_workspace_bytes(M, K) bytes, needed if
 *   dweight or dbias is given.
 * Shape rules as layer_norm_forward.
 */
size_t layer_norm_backward_workspace_bytes(int64_t M, int64_t K);
w8a8_status layer_norm_backward(w8a8_dtype xt, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                const float *mean, const float *rstd, int64_t M, int64_t K, w8a8_dtype wt,
                                const void *weight, void *dx, int64_t lddx, float *dweight, float *dbias,
                                void *workspace, hipStream_t stream);

/*
 * Row-wise activation quantization (w8a8_quant_act_rowwise) of the rows'
 * layer norm, in one pass: the shared absmax rule on the f32 values of y
 * (never rounded to bf16).  A NaN in a row's y makes its absmax and so its
 * scale NaN, e4m3's codes too; beside an infinite scale e4m3's codes are zeros
 * of y's signs, NaN where y is infinite.  int8 codes are 0 beside a scale that
 * is not finite (a product with either is NaN).
 *   x [M, ldx] of type xt; weight, bias, eps, mean, rstd as
 *   layer_norm_forward; xq codes [M, ldq], columns K .. ldq - 1 written as
 *   zero; x_scale f32 [M].
 * Shape rules as layer_norm_forward, and ldq >= K, ldq % 16 == 0,
 * ldq <= 2^24.
 */
w8a8_status w8a8_quant_act_rowwise_layer_norm(w8a8_qtype qtype, w8a8_dtype xt, const void *x, int64_t M, int64_t K,
                                              int64_t ldx, w8a8_dtype wt, const void *weight, const void *bias,
                                              float eps, void *xq, int64_t ldq, float *x_scale, float *mean,
                                              float *rstd, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_BLOCK_H_ */
