/*
 * w8a8_experts.h -- the microscaled 4-bit format (quantizers, dequantizer,
 * product) and products whose rows fall into groups with a weight each: the
 * experts of a mixture, in 8 bits and in the 4-bit format, with their input
 * gradients.
 *
 * Ownership, execution and errors are those of w8a8.h: device pointers owned
 * by the caller, arguments checked on the host before anything is launched,
 * kernels enqueued on `stream` without allocation, clearing or
 * synchronization (graph-capturable), sizes of 0 a successful no-op, base
 * pointers 16-byte aligned.  An output overlaps no other argument.  Results do
 * not depend on the order in which workgroups run (no atomics): the same call
 * gives the same bits.
 */
#ifndef W8A8_EXPERTS_H_
#define W8A8_EXPERTS_H_

#include "w8a8_block.h" /* w8a8_dtype */

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------ the microscaled 4-bit format
 *
 * OCP Microscaling Formats (MX) v1.0, MXFP4.  A block of 32 values along a row
 * shares a scale 2^e, held as the byte e + 127 (E8M0; 255 is NaN); a value is
 * an E2M1 code of 4 bits: sign, then the index of its magnitude among
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   e = max(floor(log2(absmax of the block)) - 2, -127); code = x / 2^e
 *   rounded to the nearest magnitude, ties to the even code, at most 6.
 * A block that holds an infinity or a NaN gets the scale byte 255 and codes 0:
 * all of its 32 values read as NaN.
 *
 * Layout of a matrix of R rows and `ldq` columns (ldq % 32 == 0): codes
 * [R, ldq / 2], two a byte, the even column in the low half; scales
 * [R, mxfp4_scale_stride(ldq)] bytes, the row's ldq / 32 and padding up to a
 * multiple of 16.  The quantizers write the padding as 127; nothing reads it.
 */

/* 16 * ceil(ldq / 512): bytes from one row's scales to the next one's. */
int64_t mxfp4_scale_stride(int64_t ldq);

/*
 * Quantizes the rows of x [M, ldx] (first K columns, type xt), blocks along K.
 * Columns K .. ldq - 1 of the codes are written as 0.
 * Shape rules: 0 <= M <= 2^30; 1 <= K <= 2^22; K <= ldx <= 2^24, any alignment
 * of the rows; K <= ldq <= 2^22, ldq % 32 == 0; M * ceil(ldq / 512) <= 2^27.
 */
w8a8_status mxfp4_quantize(w8a8_dtype xt, const void *x, int64_t M, int64_t K, int64_t ldx, uint8_t *xq, int64_t ldq,
                           uint8_t *xs, hipStream_t stream);

/*
 * Quantizes the transposes of B matrices w [B, N, K] (type xt, rows ldx apart,
 * matrices N * ldx apart): codes [B, K, ldq / 2], scales
 * [B, K, mxfp4_scale_stride(ldq)] of the K rows of N values each, blocks along
 * N.  What the input gradient's product takes as its weight.
 * Shape rules: 0 <= B <= 65535; 1 <= N, K <= 2^22; K <= ldx <= 2^24;
 * N <= ldq <= 2^22, ldq % 32 == 0; B * N * ldx <= 2^40; fewer than 2^24 tiles
 * of 256 x 64: B * 2 ceil(ldq / 512) * ceil(K / 64).
 */
w8a8_status mxfp4_quantize_transposed(w8a8_dtype xt, const void *w, int64_t B, int64_t N, int64_t K, int64_t ldx,
                                      uint8_t *wq, int64_t ldq, uint8_t *ws, hipStream_t stream);

/*
 * y[m, k] = value of the code (type yt, first K columns of rows ldy apart):
 * exact in either type wherever it is in range (beyond f32's range: infinite).
 * Shape rules as mxfp4_quantize.
 */
w8a8_status mxfp4_dequantize(const uint8_t *xq, const uint8_t *xs, int64_t M, int64_t K, int64_t ldq, w8a8_dtype yt,
                             void *y, int64_t ldy, hipStream_t stream);

/*
 * y[m, n] = bf16(sum_k x[m, k] * w[n, k] + bias[n]): codes of x [M, K] and
 * w [N, K] in the format above with ldq = K, f32 sums, one rounding.
 *   bias bf16 [N] or NULL; y bf16 [M, N].
 * Shape rules: 0 <= M, N <= 2^30; 32 <= K <= 2^22, K % 32 == 0; at most 2^31 - 1
 * tiles of 16 x 16.
 */
w8a8_status mxfp4_linear(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                         const uint16_t *bias, int64_t M, int64_t N, int64_t K, uint16_t *y, hipStream_t stream);

/*
 * dX = dY . W of mxfp4_linear: dyq, dys [M, N] quantized along N, wq_t, ws_t
 * the transposed weight [K, N] (mxfp4_quantize_transposed).  N % 32 == 0: pad
 * both with ldq where the layer's width is no multiple.
 */
w8a8_status mxfp4_linear_backward_dx(const uint8_t *dyq, const uint8_t *dys, const uint8_t *wq_t, const uint8_t *ws_t,
                                     int64_t M, int64_t N, int64_t K, uint16_t *dx, hipStream_t stream);

/* ------------------------------------------------------- products of groups
 *
 * The M rows of the output fall into E groups, one after the other: group g
 * has the rows offsets[g] .. offsets[g + 1] - 1 (offsets: E + 1 int32 on the
 * device, as routing leaves them; the host does not see them).  Row p takes
 * row t = rows[p] of x (int32 [M] on the device, or NULL: t = p), so that
 * tokens sent to several experts are quantized and stored once:
 *   y[p, n] = bf16(x_scale[t] * w_scale * sum_k x[t, k] * w[g, n, k] + bias[g, n])
 * Rows in no group (before offsets[0], from offsets[E] on) are not written.
 * Groups may be empty.  Offsets are clamped to [0, M], and one below an
 * earlier one counts as that; a row index outside [0, X) reads as a row of
 * zeros: nothing is read or written out of range, whatever they hold.
 *   xq codes [X, K], x_scale f32 [X]; wq codes [E, N, K], w_scale f32 [E], or
 *   [E, N] with per_channel; bias bf16 [E, N] or NULL; y bf16 [M, N].
 * Sums of int8 products are int32: exact while K < 2^17, whatever the codes,
 * and modulo 2^32 beyond.  Sums of e4m3 products are f32, but before it adds
 * them the matrix unit lines the products of eight neighbouring codes (k = 8 c
 * .. 8 c + 7) up with the greatest of the eight and cuts them off 13 bits below
 * its leading bit.  A term is thus off by less than 2^-13 of the greatest of its
 * eight, and not at all from 2^-5 of it on (a product has 8 bits).  On normal
 * values y differs by 2e-4 from that of f32 sums (relative Frobenius error) and
 * is as far from the exact product as that one is, 1.7e-3, bf16's rounding.
 * Shape rules: 0 <= M, N, X <= 2^30 (X = M if rows is NULL); 16 <= K <= 2^22,
 * K % 16 == 0; 1 <= E <= 4096; with rows, X * K <= 2^31 (bytes of codes); at
 * most 2^31 - 1 tiles: (M / 16 + E) * ceil(N / 16).
 */
w8a8_status w8a8_linear_grouped(w8a8_qtype qtype, const void *xq, int64_t X, const float *x_scale, const void *wq,
                                const float *w_scale, int per_channel, const uint16_t *bias, const int32_t *offsets,
                                int64_t E, const int32_t *rows, int64_t M, int64_t N, int64_t K, uint16_t *y,
                                hipStream_t stream);

/*
 * dX[p, :] = dY[p, :] . W[g] from dyq codes [M, N], dy_scale f32 [M] and the
 * transposed codes wq_t [E, K, N] with w_scale f32 [E]; dx bf16 [M, K], in the
 * groups' order (the rows of one token are the caller's to add up).
 * A forward call's scale for each channel does not leave this sum: multiply
 * dY[p, n] by w_scale[g, n] before it is quantized, and pass scales of 1.
 * Shape rules as the forward call's with N and K exchanged.
 */
w8a8_status w8a8_linear_grouped_backward_dx(w8a8_qtype qtype, const void *dyq, const float *dy_scale,
                                            const void *wq_t, const float *w_scale, const int32_t *offsets, int64_t E,
                                            int64_t M, int64_t N, int64_t K, uint16_t *dx, hipStream_t stream);

/*
 * The same in the 4-bit format: xq, xs [X, K], wq [E, N, K / 2], ws
 * [E, N, mxfp4_scale_stride(K)]; no other scales.  Sums are f32 (eight
 * neighbouring products share their scales and fit the 13 bits).
 * K % 32 == 0; with rows, X * K / 2 <= 2^31.
 */
w8a8_status mxfp4_linear_grouped(const uint8_t *xq, int64_t X, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                                 const uint16_t *bias, const int32_t *offsets, int64_t E, const int32_t *rows,
                                 int64_t M, int64_t N, int64_t K, uint16_t *y, hipStream_t stream);

/* dyq, dys [M, N]; wq_t, ws_t [E, K, N] (mxfp4_quantize_transposed); N % 32 == 0. */
w8a8_status mxfp4_linear_grouped_backward_dx(const uint8_t *dyq, const uint8_t *dys, const uint8_t *wq_t,
                                             const uint8_t *ws_t, const int32_t *offsets, int64_t E, int64_t M,
                                             int64_t N, int64_t K, uint16_t *dx, hipStream_t stream);

/*
 * Diagnostic: which kernel a product of M rows in E groups takes on the current
 * device (type 0 int8, 1 e4m3, 2 the 4-bit format; E = 1 for mxfp4_linear), so
 * that a test can tell what a shape exercises: 0 .. 3 tiles of 16 x 16, 16 x
 * 32, 32 x 32, 64 x 64 with operands staged by each wave; 4 and 5 128 x 128
 * with a ring of four and of two stages; 6 256 x 256; 7 256 x 256 for whole
 * rounds over the chip, and a rest of at most half a round in 128 x 128.  -1 for
 * sizes below 1 or another type.  Enqueues nothing.
 */
int w8a8_probe_grouped_kernel(int type, int64_t M, int64_t N, int64_t K, int64_t E);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_EXPERTS_H_ */
