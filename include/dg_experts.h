/*
 * dg_experts.h - C ABI of the steps of an expert layer for many tokens around
 * the contiguous-grouped products of dg_fp8.h and dg_int8.h:
 *
 *   dg_moe_topk -> dg_moe_dispatch_* -> grouped product -> dg_swiglu_quantize_*
 *               -> grouped product -> dg_moe_unpermute
 *
 * and the gradients of the steps here.  Same library, same conventions as
 * dg_ops.h: device pointers to caller-owned, contiguous, row-major memory
 * aligned to 16 bytes; work is enqueued on `stream` and no call synchronizes;
 * arguments are checked on the host, sizes first, then pointers, before
 * anything is enqueued; workspaces as there; outputs overlap no input.  Sums
 * are taken in a fixed order without atomics: the same inputs give the same
 * bits.
 */
#ifndef DG_EXPERTS_H
#define DG_EXPERTS_H

#include "dg_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Places of tokens sorted by expert, each expert's rows padded to 128.
 *   ids     [T][k] int32: the experts of each token; a value outside [0, E) is
 *           an expert elsewhere, and an expert may appear more than once in a row
 *   rows    [T][k] int32 (output): the sorted row of each pair, -1 elsewhere
 *   layout  [M] int32 (output): the expert of each sorted row, -1 for padding
 *           and for the rows behind the last expert's: a grouped_layout
 *   offsets [E + 1] int32 (output): first row of each expert; the last is the
 *           number of rows up to the end of the last expert's padding
 * Expert e's rows start at offsets[e], hold its pairs in the order of the
 * tokens (and of k within one), and end on a multiple of 128; an expert
 * without pairs takes no rows.  M is at least what dg_moe_sort_rows gives: the
 * most rows that any choice of experts needs.  T = 0 writes an empty plan (ids
 * and rows may then be NULL).
 * Sizes: 0 <= T, 1 <= k <= 64, T * k <= 2^30, 1 <= E <= 4096, M a multiple of
 * 128 below 2^31. */
dg_status dg_moe_sort(const int32_t* ids, int32_t* rows, int32_t* layout, int32_t* offsets,
                      int64_t T, int64_t k, int64_t E, int64_t M, void* workspace,
                      int64_t workspace_bytes, void* stream);
/* The most sorted rows that T tokens of k choices among E experts can need:
 * T k + 127 min(E, T k), rounded down to a multiple of 128; into *rows (host
 * memory).  DG_ERR_SHAPE where that is 2^31 or more. */
dg_status dg_moe_sort_rows(int64_t T, int64_t k, int64_t E, int64_t* rows);
/* Bytes of workspace for dg_moe_sort and the dispatch calls, into *bytes (host
 * memory). */
dg_status dg_moe_sort_workspace(int64_t T, int64_t k, int64_t E, int64_t* bytes);

/* Sorting and copying in one call: token t's activations go into the row of
 * each of its pairs.  ids, rows, layout, offsets, T, k, E, M and the workspace
 * as in dg_moe_sort.
 *   x    [T][H] bf16 bits
 *   out  [M][H] bf16 bits (output); rows of padding, and those behind the last
 *        expert's, are set to zero
 * or quantized once per token on the way, rows of padding left as they were:
 *   q    [M][H] e4m3 codes, s [M][H/128] fp32    (_fp8: dg_quantize_fp8_per_token's recipe)
 *   q    [M][H] e4m3 codes, s [M][SP] E8M0 bytes (_fp8_e8m0: dg_quantize_fp8_per_token_e8m0's;
 *        SP = H/128 rounded up to a multiple of 4, padding bytes left as they were)
 *   q    [M][H] int8, s [M] fp32                 (_int8: dg_quantize_int8_per_row's)
 * A block (int8: a row) that holds a NaN or an infinity gets the scale NaN
 * (byte 255), which makes its rows of the product NaN.
 * Sizes as dg_moe_sort; H a multiple of 8, for the quantized forms of 128, and
 * below 2^24. */
dg_status dg_moe_dispatch(const uint16_t* x, const int32_t* ids, uint16_t* out, int32_t* rows,
                          int32_t* layout, int32_t* offsets, int64_t T, int64_t k, int64_t E,
                          int64_t H, int64_t M, void* workspace, int64_t workspace_bytes,
                          void* stream);
dg_status dg_moe_dispatch_fp8(const uint16_t* x, const int32_t* ids, uint8_t* q, float* s,
                              int32_t* rows, int32_t* layout, int32_t* offsets, int64_t T,
                              int64_t k, int64_t E, int64_t H, int64_t M, void* workspace,
                              int64_t workspace_bytes, void* stream);
dg_status dg_moe_dispatch_fp8_e8m0(const uint16_t* x, const int32_t* ids, uint8_t* q, uint8_t* s,
                                   int32_t* rows, int32_t* layout, int32_t* offsets, int64_t T,
                                   int64_t k, int64_t E, int64_t H, int64_t M, void* workspace,
                                   int64_t workspace_bytes, void* stream);
dg_status dg_moe_dispatch_int8(const uint16_t* x, const int32_t* ids, int8_t* q, float* s,
                               int32_t* rows, int32_t* layout, int32_t* offsets, int64_t T,
                               int64_t k, int64_t E, int64_t H, int64_t M, void* workspace,
                               int64_t workspace_bytes, void* stream);

/* Sorted rows back to their tokens, weighted.
 *   y       [M][H] bf16 bits     rows [T][k] int32 as dg_moe_sort makes them
 *   weights [T][k] fp32, or NULL for ones (which gives the gradient of
 *           dg_moe_dispatch with respect to x)
 *   out     [T][H] bf16 bits (output, every row written)
 *   out[t] = bf16( sum over j of weights[t][j] * y[rows[t][j]] ), in fp32 in
 * the order of j; entries of rows outside [0, M) add nothing, whatever their
 * weight.  Sizes: T, M >= 0, T and M below 2^31, 1 <= k <= 64, H a multiple of
 * 8 below 2^24. */
dg_status dg_moe_unpermute(const uint16_t* y, const int32_t* rows, const float* weights,
                           uint16_t* out, int64_t T, int64_t k, int64_t H, int64_t M, void* stream);

/* Gradients of dg_moe_unpermute.
 *   grad         [T][H] bf16 bits: the gradient of out
 *   layout       [M] int32 or NULL: as dg_moe_sort makes it together with rows, so
 *                that an entry of rows names every row whose entry here is not
 *                negative
 *   grad_y       [M][H] bf16 bits (output) or NULL when not wanted:
 *                grad_y[rows[t][j]] = bf16(weights[t][j] * grad[t]); with layout,
 *                rows whose entry is negative are set to zero; other rows that no
 *                entry of `rows` names are left as they were (a caller that drops
 *                a pair by writing -1 into rows writes -1 into its row's layout
 *                entry too, or clears grad_y itself and gives no layout)
 *   grad_weights [T][k] fp32 (output) or NULL when not wanted (y may then be
 *                NULL): the sum over H of grad[t] * y[rows[t][j]], 0 where
 *                rows[t][j] is outside [0, M)
 * No two entries of rows that are in [0, M) may be the same (dg_moe_sort makes
 * none; which of two gradients such a row would get is not defined).  At least
 * one output is not NULL.  Sizes as dg_moe_unpermute. */
dg_status dg_moe_unpermute_backward(const uint16_t* grad, const uint16_t* y, const int32_t* rows,
                                    const float* weights, const int32_t* layout, uint16_t* grad_y,
                                    float* grad_weights, int64_t T, int64_t k, int64_t H, int64_t M,
                                    void* stream);

/* The gate between an expert's two products: h = silu(gate) * up, in fp32,
 * (gate, up) = the halves of a row.  A sigmoid below 2^-126 (gates below -87.3)
 * may come as 0, here and in the gradient.
 *   z       [M][2I] bf16 bits: the first product's rows
 *   layout  [M] int32, or NULL for every row: rows whose entry is negative are
 *           not computed
 *   h       [M][I] bf16 bits (output), or quantized without a rounding between:
 *   q, s    as in the dispatch calls, with I in the place of H (outputs)
 * Rows not computed are set to zero in h and left as they were in q and s.
 * Sizes: 0 <= M < 2^31, I a multiple of 8, for the quantized forms of 128,
 * below 2^23. */
dg_status dg_swiglu(const uint16_t* z, const int32_t* layout, uint16_t* h, int64_t M, int64_t I,
                    void* stream);
dg_status dg_swiglu_quantize_fp8(const uint16_t* z, const int32_t* layout, uint8_t* q, float* s,
                                 int64_t M, int64_t I, void* stream);
dg_status dg_swiglu_quantize_fp8_e8m0(const uint16_t* z, const int32_t* layout, uint8_t* q,
                                      uint8_t* s, int64_t M, int64_t I, void* stream);
dg_status dg_swiglu_quantize_int8(const uint16_t* z, const int32_t* layout, int8_t* q, float* s,
                                  int64_t M, int64_t I, void* stream);

/* Gradient of the gate with respect to z, recomputed from z:
 *   p = sigmoid(gate);  grad_gate = grad_h * up * p * (1 + gate * (1 - p)),
 *   grad_up = grad_h * gate * p, in fp32, rounded once.
 *   grad_h [M][I] bf16 bits     grad_z [M][2I] bf16 bits (output; rows whose
 *   layout entry is negative are set to zero)
 * Sizes as dg_swiglu. */
dg_status dg_swiglu_backward(const uint16_t* z, const uint16_t* grad_h, const int32_t* layout,
                             uint16_t* grad_z, int64_t M, int64_t I, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DG_EXPERTS_H */
