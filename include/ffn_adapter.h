/*
 * ffn_adapter.h -- C ABI of low-rank adapters beside a shared projection
 * (MI355X / gfx950), part of the same library as ffn_sparse.h: the rows of many
 * requests (or sequences of a training batch), each with an adapter of its own
 * or none, through their adapters at once, and the gradients.
 *
 * Conventions are those of ffn_linear.h: device pointers allocated by the
 * caller, 16-byte aligned, row-major dense; calls are asynchronous on `stream`,
 * check their arguments before launching anything, write nothing on an error,
 * allocate nothing, keep no state and may be captured into a graph. A call
 * without rows does nothing but what is said below, and takes null pointers. An
 * output shares memory with an input only where that is said.
 *
 * Rows. `offsets` (device, int32 [groups + 1]) and `rows` (device, NULL or int32
 * [m]) say which rows an adapter has: places offsets[g] .. offsets[g + 1] - 1
 * are adapter g's, and place p is row rows[p], or row p without `rows`
 * (ffn_group_rows of ffn_experts.h makes both from the adapter of each row).
 * Places before offsets[0] and from offsets[groups] on have no adapter. Offsets
 * outside 0..m are taken as the nearest of the two, one below an earlier one as
 * that one. `rows` names every row once; a place whose row is outside 0 .. m - 1
 * is left out.
 *
 * Sums are held in fp32 and made in a fixed order; x A^T and dy B are kept in
 * fp32 between the two products and enter the second as the sum of two bf16
 * numbers (three where the output is fp32), which hold them to 2^-16 (2^-24) of
 * their size. An infinity or a NaN makes what it enters infinite or NaN (which of
 * the two, the parts decide: an infinite weight times a part that is 0 is NaN), and
 * nothing else; what rows without an adapter and adapters without rows hold does
 * not matter.
 */
#ifndef FFN_ADAPTER_H
#define FFN_ADAPTER_H

#include <stddef.h>
#include <stdint.h>

#include "ffn_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FFN_ADAPTER_ABI_VERSION 1
#define FFN_ADAPTER_MAX_GROUPS 1024
#define FFN_ADAPTER_MAX_RANK 256

int32_t ffn_adapter_abi_version(void);

/* Bytes of workspace ffn_adapter_forward needs (0: none, as for few rows, or invalid). */
size_t ffn_adapter_forward_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t r, int32_t groups);

/* y[t] = base[t] + scales[g] B_g (A_g x[t]) for the rows t of each adapter g,
 * y[t] = base[t] for the others.
 *   x       [m x k] bf16; a [groups x r x k] bf16; b [groups x n x r] bf16
 *   scales  NULL (ones) or [groups] fp32
 *   base    NULL (zeros) or [m x n] of y_dtype: the shared projection's output
 *   y       [m x n] of y_dtype (FFN_F32 or FFN_BF16), written in full; base
 *           itself: added to in place, rows without an adapter not touched
 * m: up to 2^26. n, k: multiples of 8, up to 2^22. r: multiple of 8, 8 .. FFN_ADAPTER_MAX_RANK
 * (an adapter of lower rank has zeros behind it). 1 <= groups <=
 * FFN_ADAPTER_MAX_GROUPS. */
ffn_status ffn_adapter_forward(const void *x, const void *a, const void *b, const float *scales,
                               const int32_t *offsets, const int32_t *rows, int32_t groups, int32_t m, int32_t n,
                               int32_t k, int32_t r, const void *base, void *y, int32_t y_dtype, void *workspace,
                               size_t workspace_bytes, void *stream);

/* Bytes of workspace ffn_adapter_backward needs (0 if invalid, or without rows). */
size_t ffn_adapter_backward_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t r, int32_t groups);

/* Gradients of <dy, y> (that of base is dy itself).
 *   dy    [m x n] bf16
 *   base  NULL (zeros) or [m x k] bf16: the shared projection's gradient of x
 *   dx    NULL or [m x k] bf16: base[t] + scales[g] A_g^T (B_g^T dy[t]), base[t] for
 *         rows without an adapter; may be base itself, as above
 *   da    NULL or [groups x r x k] fp32: scales[g] sum over its rows of (B_g^T dy) x^T
 *   db    NULL or [groups x n x r] fp32: scales[g] sum over its rows of dy (A_g x)^T
 *         both written (zeros for an adapter without rows) or, with accumulate = 1,
 *         added to
 * One of dx, da and db at least. x may be NULL without da and db, a without dx
 * and db, b without dx and da; base has to be NULL without dx. With m = 0, da
 * and db are cleared unless they accumulate. */
ffn_status ffn_adapter_backward(const void *x, const void *a, const void *b, const float *scales, const void *dy,
                                const int32_t *offsets, const int32_t *rows, int32_t groups, int32_t m, int32_t n,
                                int32_t k, int32_t r, const void *base, void *dx, float *da, float *db,
                                int32_t accumulate, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FFN_ADAPTER_H */
