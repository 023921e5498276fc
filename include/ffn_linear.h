/*
 * ffn_linear.h -- C ABI of the operators around the FFN (MI355X / gfx950),
 * part of the same library as ffn_sparse.h: RMS norm with the residual's
 * addition, 8-bit blocks with a scale each, the matrix product of such blocks,
 * and matrix products grouped by expert, with what their backward passes need.
 *
 * Conventions (as in ffn_sparse.h): device pointers allocated by the caller,
 * 16-byte aligned; row-major dense matrices; every call is asynchronous on
 * `stream` (a hipStream_t of the current device, NULL = the null stream),
 * checks its arguments before launching anything and writes nothing on an
 * error; the library never allocates device memory and never synchronises.
 * The calls keep no state: any number of them may run at once, on any
 * streams, as long as no two of them share a workspace or an output. All may
 * be captured into a graph. A call with no rows (m = 0) does nothing but what
 * is said below, and takes null pointers. FFN_E_HIP reports a failed launch.
 * `dtype` is ffn_dtype (FFN_F32 or FFN_BF16); sums are held in fp32 (those of
 * ffn_fp8_linear for a bf16 output with an exception, said there), so rows
 * whose squares pass its range have an infinite mean. m is at most 2^31 - 2^16.
 *
 * 8-bit blocks. A matrix [m x k] held in 8 bits is
 *   q      uint8 [m x k]: e4m3 (OCP; 1 sign, 4 exponent and 3 mantissa bits,
 *          largest value 448, no infinities)
 *   scale  fp32, one for each block; a value is q * scale.
 *          block_rows = 1:   blocks of 1 x 128,   scale [ceil(k/128) x m]
 *          block_rows = 128: blocks of 128 x 128, scale [ceil(m/128) x ceil(k/128)]
 * The last blocks of a row or column may be shorter. A block's scale is
 * max(max|x| * fp32(1/448), 2^-100), q = x * (1 / scale) in fp32, rounded to
 * nearest even. A block that holds an infinity or a NaN has an infinite or NaN
 * scale and stands for no number anywhere: its products are NaN.
 *
 * Experts. `offsets` (device, int32 [groups + 1], non-decreasing, from 0 to m)
 * gives the rows of each expert: rows offsets[g] .. offsets[g + 1] - 1 belong
 * to expert g, which may have none. It is read on the device, so routing needs
 * no host copy. Rows before offsets[0] and from offsets[groups] on belong to
 * no expert: they are not read, and those of the output are left as they were.
 * Offsets outside 0..m are taken as the nearest of the two, one below an
 * earlier one as that one, so whatever they hold no row has two experts.
 */
#ifndef FFN_LINEAR_H
#define FFN_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#include "ffn_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FFN_LINEAR_ABI_VERSION 1
#define FFN_LINEAR_MAX_GROUPS 256

int32_t ffn_linear_abi_version(void);

/* RMS norm: r = x + residual (rounded to dtype), y = r * rstd * w with
 * rstd = 1 / sqrt(mean(r^2) + eps), per row.
 *   x         [m x d]; residual NULL or [m x d] (then r_out is required)
 *   w         [d]
 *   r_out     NULL or [m x d] dtype: r, the residual stream that goes on (may be x
 *             or residual itself)
 *   y         NULL or [m x d] dtype
 *   q, scale  NULL or y in 8 bits, blocks of 1 x 128, rounded from fp32 once
 * One of y and q at least. d: multiple of 8, 8..16384. eps >= 0, finite. */
ffn_status ffn_rmsnorm_forward(const void *x, const void *residual, const void *w, int32_t dtype,
                               int32_t m, int32_t d, float eps, void *r_out, void *y, uint8_t *q,
                               float *scale, void *stream);

/* Bytes of workspace ffn_rmsnorm_backward needs (0 if invalid). */
size_t ffn_rmsnorm_backward_workspace_bytes(int32_t m, int32_t d);

/* Gradients of <dy, y> + <dr, r> of the norm above:
 *   dx = rstd (w dy - h mean(w dy h)) + dr with h = r rstd (the gradient of x
 *   and of the residual alike), dw = sum over the rows of dy h.
 *   r, dy     [m x d] dtype: the normalised rows, the gradient of y
 *   dr        NULL or [m x d] dtype: the gradient that reaches r besides
 *   dx        NULL or [m x d] dtype (may be dy or dr itself)
 *   dw        NULL or [d] fp32: written, or added to if accumulate is 1
 * One of dx and dw at least. With m = 0, dw is cleared unless it accumulates.
 * The rows are summed in a fixed order: dw is the same from run to run. */
ffn_status ffn_rmsnorm_backward(const void *r, const void *w, const void *dy, const void *dr, int32_t dtype,
                                int32_t m, int32_t d, float eps, void *dx, float *dw, int32_t accumulate,
                                void *workspace, size_t workspace_bytes, void *stream);

/* x [groups x m x k] (dtype) in 8 bits, each of the `groups` matrices by itself.
 *   q, scale    [groups x m x k] and its scales, one such array for each matrix
 *   qt, scale_t NULL, or the transposed matrices [groups x k x mt], mt = m rounded
 *               up to a multiple of 16 (the added columns hold zeros), and their
 *               scales: of blocks of 1 x 128, that is of 128 rows of x
 *               (block_rows = 1: [groups x ceil(m/128) x k]), or the same blocks of
 *               128 x 128 (block_rows = 128: [groups x ceil(k/128) x ceil(m/128)])
 * k: multiple of 16. block_rows: 1 or 128. Fewer than 2^24 tiles of 128 x 128 in
 * all, begun ones counted (FFN_E_UNSUPPORTED otherwise). */
ffn_status ffn_fp8_quantize(const void *x, int32_t dtype, int32_t groups, int32_t m, int32_t k,
                            int32_t block_rows, uint8_t *q, float *scale, uint8_t *qt, float *scale_t,
                            void *stream);

/* Bytes of workspace ffn_fp8_linear may use for this shape (0: none, or invalid). */
size_t ffn_fp8_linear_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t groups);

/* y = x w^T of 8-bit blocks: y[t, i] = sum over the blocks b of k of
 * x_scale[b, t] w_scale[., b] sum_{j in b} x[t, j] w[i, j].
 *   x, x_scale  [m x k], blocks of 1 x 128
 *   w, w_scale  [n x k], blocks of w_block_rows x 128 (1 or 128); with offsets
 *               one matrix and scale array for each expert: [groups x n x k],
 *               w_block_rows 128
 *   offsets     NULL (one product, groups = 1), or the rows of each expert
 *   y           [m x n] of y_dtype; accumulate = 1 adds to it (FFN_F32 only)
 *   workspace   NULL, or ffn_fp8_linear_workspace_bytes of scratch (a smaller
 *               one is not used): with it, small products are cut along k
 * y_dtype also says how the sums are made. FFN_F32: every product x[t, j] w[i, j]
 * is exact and they are added in fp32. FFN_BF16: on the e4m3 matrix instructions,
 * twice as fast, which hold the sum of 8 products (8 consecutive j, from a multiple
 * of 8 on) to 13 bits below the largest of them: each other product of the eight
 * loses less than 2^-13 of the largest, so an output is off by up to 7 * 2^-13 of
 * the largest product of each eight (scaled, summed over the eights) besides its
 * rounding. That is about 2e-5 of a product of normal values, 6e-5 with a few
 * channels 20 times as large; where large products cancel it can be all that is
 * left of an output (2^16 - 2^16 + 2^2 in one eight may come out as 0): take FFN_F32.
 * A block's sum is multiplied by the product of its two scales, which is made in
 * fp32 and has to lie in 2^-126 .. 2^128 unless one of the blocks holds zeros only
 * (of blocks from ffn_fp8_quantize: max|x| max|w| in 2^-108 .. 2^145): above, the
 * output is infinite, or NaN where the block's sum is 0; below, it loses bits.
 * k: multiple of 16; n, k <= 2^22. Also the backward pass: dx = dy w is the product of dy's
 * blocks with the transposed w, dw = dy^T x the product of dy's and x's
 * transposed blocks (w_block_rows = 1), all from ffn_fp8_quantize. */
ffn_status ffn_fp8_linear(const uint8_t *x, const float *x_scale, const uint8_t *w, const float *w_scale,
                          int32_t w_block_rows, int32_t m, int32_t n, int32_t k, const int32_t *offsets,
                          int32_t groups, void *y, int32_t y_dtype, int32_t accumulate, void *workspace,
                          size_t workspace_bytes, void *stream);

/* Bytes of workspace ffn_grouped_forward may use for this shape (0: none, or invalid). */
size_t ffn_grouped_forward_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t groups);

/* y[t] = W_g x[t] for the rows t of each expert g, bf16.
 *   x [m x k] bf16; w [groups x n x k] bf16; offsets as above (required)
 *   y [m x n] of y_dtype
 *   workspace   as for ffn_fp8_linear
 * n, k: multiples of 8, up to 2^22 as in ffn_fp8_linear. 1 <= groups <= FFN_LINEAR_MAX_GROUPS. */
ffn_status ffn_grouped_forward(const void *x, const void *w, const int32_t *offsets, int32_t groups, int32_t m,
                               int32_t n, int32_t k, void *y, int32_t y_dtype, void *workspace,
                               size_t workspace_bytes, void *stream);

/* Bytes of workspace ffn_grouped_backward may use for this shape (0: none, or invalid). */
size_t ffn_grouped_backward_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t groups);

/* Gradients of <dy, y> of the product above.
 *   dy [m x n] bf16
 *   dx NULL or [m x k] bf16: dx[t] = W_g^T dy[t]
 *   dw NULL or [groups x n x k] fp32: dW_g = sum over the rows t of g of
 *      dy[t] x[t]^T, written (zeros for an expert without rows) or, with
 *      accumulate = 1, added to
 *   workspace as for ffn_fp8_linear
 * One of dx and dw at least; x may be NULL without dw, w without dx. With m = 0,
 * dw is cleared unless it accumulates. Sums run in a fixed order. */
ffn_status ffn_grouped_backward(const void *x, const void *w, const void *dy, const int32_t *offsets,
                                int32_t groups, int32_t m, int32_t n, int32_t k, void *dx, float *dw,
                                int32_t accumulate, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FFN_LINEAR_H */
