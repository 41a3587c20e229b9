/*
 * dg_int8.h - C ABI of the 8-bit integer products: operands in int8 with one
 * fp32 scale per row on either side (per token for the activations, per output
 * channel for the weights).  Same library, same conventions as dg_fp8.h;
 * outputs overlap no input.
 *
 *   D[m,n] = bf16( (sa[m] * sb[n]) * sum_k A[m,k] * B[n,k] )
 *
 * A and B are K-contiguous.  The sum over k is exact, in 32-bit integers; it is
 * rounded to fp32 once, as is the product of the scales, and the result of
 * their multiplication to bf16.
 */
#ifndef DG_INT8_H
#define DG_INT8_H

#include "dg_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Dense form.
 *   A  [M][K]  int8     sa [M] fp32
 *   B  [N][K]  int8     sb [N] fp32
 *   D  [M][N]  bf16 bits (output)
 * Sizes: as dg_fp8_gemm_nt, and K < 2^17 (2^17 products of -128 by -128 would
 * pass the largest int32). */
dg_status dg_int8_gemm_nt(const int8_t* A, const float* sa, const int8_t* B, const float* sb,
                          uint16_t* D, int64_t M, int64_t N, int64_t K, void* stream);

/* Contiguous-grouped form (expert weights, rows sorted by expert).
 *   A  [M_sum][K] int8   sa [M_sum] fp32
 *   B  [G][N][K]  int8   sb [G][N] fp32
 *   D  [M_sum][N] bf16 bits    grouped_layout [M_sum] int32
 * Rows and blocks as in dg_fp8_gemm_grouped_contiguous: M_sum % 128 == 0, row
 * r is computed with B[g], sb[g] for g = grouped_layout[r] in [0, G), any
 * other row is not written, and a block of 128 rows that carries several ids
 * is computed once per id.  Sizes: as there, and K < 2^17. */
dg_status dg_int8_gemm_grouped_contiguous(const int8_t* A, const float* sa, const int8_t* B,
                                          const float* sb, uint16_t* D,
                                          const int32_t* grouped_layout, int64_t M_sum, int64_t N,
                                          int64_t K, int64_t G, void* stream);

/* Quantization with one scale per row: x [M][K] fp32 or bf16 bits -> q [M][K]
 * int8 and s [M] fp32.  scale = amax / 127, q = x / scale rounded to the
 * nearest integer, ties to even (both divisions IEEE fp32); a row of zeros
 * stores scale 0 and codes 0.  A row that holds a NaN or an infinity gets the
 * scale NaN and codes 0, which makes its row (or column) of the product NaN.
 * Sizes: M >= 0, K > 0 with K % 128 == 0, K < 2^24. */
dg_status dg_quantize_int8_per_row(const float* x, int64_t M, int64_t K, int8_t* q, float* s,
                                   void* stream);
dg_status dg_quantize_int8_per_row_bf16(const uint16_t* x, int64_t M, int64_t K, int8_t* q,
                                        float* s, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DG_INT8_H */
