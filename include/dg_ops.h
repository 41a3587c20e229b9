/*
 * dg_ops.h - C ABI of the operators around the FP8 products of dg_fp8.h:
 * routing rows to experts (and the router's gradient), a whole
 * mixture-of-experts layer for a few tokens, and low-rank adapters of many
 * requests beside a shared projection.  Same library, same conventions as
 * dg_fp8.h: device pointers to caller-owned, contiguous, row-major memory
 * aligned to 16 bytes; nothing is allocated or kept between calls; work is
 * enqueued on `stream` and no call synchronizes; arguments are checked on the
 * host, sizes first, then pointers, before anything is enqueued; a call with
 * no rows (T or M equal to 0) returns DG_OK without looking at its pointers.
 * Calls that need scratch memory take a caller-owned workspace, whose size
 * the matching *_workspace function gives; its contents need no
 * initialization and mean nothing after the call.  Two calls that may run at
 * the same time need two workspaces.
 */
#ifndef DG_OPS_H
#define DG_OPS_H

#include "dg_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How router logits become scores: p = softmax of the row, or sigmoid of each logit. */
typedef enum { DG_SCORE_SOFTMAX = 0, DG_SCORE_SIGMOID = 1 } dg_scoring;

/* Router: the k experts of each token and their weights.
 *   logits  [T][E] fp32 (dg_moe_topk) or bf16 bits (dg_moe_topk_bf16)
 *   bias    [E] fp32 or NULL, added for the ranking only
 *   ids     [T][k] int32 (output), weights [T][k] fp32 (output)
 * An expert is open to a token when its logit is a number above -infinity
 * (and so is its rank); a masked expert is one with logit -infinity or NaN,
 * which counts in no softmax sum either.  rank = logit when bias is NULL and
 * n_group is 1, else p (+ bias) in 64 bits.  With n_group > 1 the experts
 * form n_group runs of E / n_group; a group's value is the sum of its two
 * best open ranks (of one if it has one), and only the topk_group best groups
 * stay open.  The k open experts of the highest rank are returned, best
 * first; ties, among groups and among experts, go to the lowest index.
 * weight = p of the expert (from the logit alone); with renormalize divided
 * by (sum of the row's k weights + 1e-20); then times `scale`.  Logits of
 * +infinity share a softmax row's whole probability equally.  Where fewer
 * than k experts are open the rest of the row is id -1, weight 0.
 * Sizes: 0 <= T <= 2^33 - 4, 1 <= E <= 1024, 1 <= k <= 64, n_group >= 1 divides E and is
 * at most 64, 1 <= topk_group <= n_group, k <= topk_group * (E / n_group). */
dg_status dg_moe_topk(const float* logits, const float* bias, int32_t* ids, float* weights,
                      int64_t T, int64_t E, int64_t k, int64_t n_group, int64_t topk_group,
                      int scoring, int renormalize, float scale, void* stream);
dg_status dg_moe_topk_bf16(const uint16_t* logits, const float* bias, int32_t* ids, float* weights,
                           int64_t T, int64_t E, int64_t k, int64_t n_group, int64_t topk_group,
                           int scoring, int renormalize, float scale, void* stream);

/* Gradient of the router's weights with respect to its logits, the choice of
 * experts held fixed.
 *   ids          [T][k] int32 as the router returned them (entries outside
 *                [0, E) and masked experts are skipped)
 *   grad_weights [T][k] fp32
 *   grad_logits  [T][E] fp32 or bf16 bits like the logits (output, every
 *                element written; masked experts get 0 whatever grad_weights
 *                holds)
 * Same scoring, renormalize and scale as the forward call.  Sizes: 0 <= T <= 2^33 - 4,
 * 1 <= E <= 1024, 1 <= k <= 64. */
dg_status dg_moe_topk_backward(const float* logits, const int32_t* ids, const float* grad_weights,
                               float* grad_logits, int64_t T, int64_t E, int64_t k, int scoring,
                               int renormalize, float scale, void* stream);
dg_status dg_moe_topk_backward_bf16(const uint16_t* logits, const int32_t* ids,
                                    const float* grad_weights, uint16_t* grad_logits, int64_t T,
                                    int64_t E, int64_t k, int scoring, int renormalize, float scale,
                                    void* stream);

/* A whole gated expert layer for a few tokens (decode).
 *   x       [T][H]     e4m3 codes     sx  [T][H/128]              fp32
 *   ids     [T][k]     int32          weights [T][k]              fp32
 *   w13     [E][2I][H] e4m3 codes     s13 [E][ceil(2I/128)][H/128] fp32
 *   w2      [E][H][I]  e4m3 codes     s2  [E][H/128][I/128]       fp32
 *   y       [T][H]     bf16 bits (output, every row written)
 * For each pair (t, j) with e = ids[t][j] in [0, E):
 *   z = x_t w13[e]^T,  h = silu(z[0..I)) * z[I..2I),
 *   h quantized by dg_quantize_fp8_per_token's recipe (one scale per 128
 *   columns), o = h w2[e]^T, all scaled as in dg_fp8.h and held in fp32;
 *   y_t = bf16(sum over j of weights[t][j] * o).
 * Other ids are experts elsewhere and add nothing; a token without any expert
 * here gets zeros.  An expert may appear more than once in a row.  A pair
 * whose hidden block holds a NaN or an infinity makes its token's row NaN.
 * Sums run in a fixed order: the same inputs give the same bits.
 * Sizes: 0 <= T <= 256 (larger batches belong to the grouped products),
 * 1 <= k <= 16, 1 <= E <= 65536, H and I multiples of 128 up to 16384. */
dg_status dg_moe_mlp_fp8(const uint8_t* x, const float* sx, const int32_t* ids, const float* weights,
                         const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2,
                         uint16_t* y, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I,
                         void* workspace, int64_t workspace_bytes, void* stream);
/* The same with E8M0 scale bytes (rows padded to a multiple of four bytes, as
 * in dg_fp8.h), the hidden activations by the power-of-two recipe. */
dg_status dg_moe_mlp_fp8_e8m0(const uint8_t* x, const uint8_t* sx, const int32_t* ids,
                              const float* weights, const uint8_t* w13, const uint8_t* s13,
                              const uint8_t* w2, const uint8_t* s2, uint16_t* y, int64_t T,
                              int64_t k, int64_t E, int64_t H, int64_t I, void* workspace,
                              int64_t workspace_bytes, void* stream);
/* Bytes of workspace for either call, into *bytes (host memory). */
dg_status dg_moe_mlp_fp8_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I,
                                   int64_t* bytes);

/* A shared projection with each row's own low-rank adapter.
 *   A, sa, B, sb, D as in dg_fp8_gemm_nt
 *   x       [M][K]    bf16 bits: the activations the adapters read
 *   lora_a  [L][R][K] bf16 bits, lora_b [L][N][R] bf16 bits, scaling [L] fp32
 *   ids     [M] int32: the row's adapter, or any value outside [0, L) for none
 *   D[m] = bf16( the dense form's sum + scaling[a] * (x_m lora_a[a]^T) lora_b[a]^T ),
 * a = ids[m], rounded once; the adapter's products are held in fp32 (the
 * rank-R vector enters its second product as a sum of two bf16 parts, 16 bits
 * of mantissa, when M is large).  Infinities and NaN give what the formula
 * gives, in their own rows.  Rows of one adapter need not be adjacent.
 * Sizes: as dg_fp8_gemm_nt, N < 2^22, K < 2^23, 1 <= L <= 65536, R a multiple
 * of 8 up to 128. */
dg_status dg_fp8_gemm_nt_lora(const uint8_t* A, const float* sa, const uint8_t* B, const float* sb,
                              uint16_t* D, const uint16_t* x, const uint16_t* lora_a,
                              const uint16_t* lora_b, const int32_t* ids, const float* scaling,
                              int64_t M, int64_t N, int64_t K, int64_t L, int64_t R,
                              void* workspace, int64_t workspace_bytes, void* stream);
/* The same with E8M0 scale bytes for the shared projection. */
dg_status dg_fp8_gemm_nt_lora_e8m0(const uint8_t* A, const uint8_t* sa, const uint8_t* B,
                                   const uint8_t* sb, uint16_t* D, const uint16_t* x,
                                   const uint16_t* lora_a, const uint16_t* lora_b,
                                   const int32_t* ids, const float* scaling, int64_t M, int64_t N,
                                   int64_t K, int64_t L, int64_t R, void* workspace,
                                   int64_t workspace_bytes, void* stream);
/* Bytes of workspace for either call, into *bytes (host memory); 0 for M = 0. */
dg_status dg_fp8_gemm_nt_lora_workspace(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R,
                                        int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* DG_OPS_H */
