// Internal launchers behind the C ABI (not exported).  Each enqueues its
// kernels on `stream` and returns DG_OK, DG_ERR_SHAPE when a size passes the
// C ABI's checks but exceeds what the kernel's grid or 32-bit offsets
// address (nothing is enqueued then), or DG_ERR_HIP when the launch fails.
// The C ABI layer has already validated sizes and pointers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_fp8.h"

namespace dg {

// Whether one dimension of a grid can be launched.  Its work-items are counted
// in 32 bits; a larger one runs only what is left of it modulo 2^32, without an
// error.
inline bool grid_fits(int64_t blocks, int64_t threads) {
    return blocks <= 0x7fffffff && blocks * threads <= 0xffffffffLL;
}

// Status of the launch just enqueued.
inline dg_status launched() { return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP; }

// DenseAcc: dense routing, D = bf16(C + A B^T scaled) with C fp32 [rows][N]
// DenseLora: dense routing, D = bf16(A B^T scaled + each row's adapter term)
enum class Form : int { Dense = 0, Contiguous = 1, Masked = 2, DenseAcc = 3, DenseLora = 4 };

// DenseLora: row m adds scaling[a] * low[m] lora_b[a]^T, a = ids[m], when a is in [0, L)
struct LoraTail {
    const float* low;        // [parts][rows][R], summed over parts
    const uint16_t* lora_b;  // bf16 [L][N][R]
    const float* scaling;    // [L]
    const int32_t* ids;      // [rows]
    int parts, L, R;         // R a multiple of 8
};

struct GemmArgs {
    const uint8_t* A;     // e4m3 codes, K-contiguous rows
    const void* sa;       // fp32 [rows][K/128]; E8M0 bytes [rows][SP] with e8m0
    const uint8_t* B;     // [groups][N][K]
    const void* sb;       // fp32 [groups][ceil(N/128)][K/128]; E8M0 [groups][ceil(N/128)][SP]
    uint16_t* D;          // bf16 bits, [rows][N]
    const int32_t* aux;   // contiguous: group id per row; masked: valid rows per group
    int64_t rows;         // dense: M; contiguous: M_sum; masked: M_max (rows per slab)
    int64_t N, K, G;
    const float* C;       // DenseAcc: fp32 [rows][N] added before the bf16 rounding
    bool e8m0 = false;    // scales are E8M0 exponent bytes, SP = K/128 rounded up to 4
    LoraTail lora = {};   // DenseLora
    bool check_only = false;  // only the checks of sizes; nothing is enqueued
};

dg_status launch_gemm(Form form, const GemmArgs& args, hipStream_t stream);

dg_status launch_quantize_per_token(const float* x, int64_t M, int64_t K, uint8_t* q, float* s,
                                     hipStream_t stream);
dg_status launch_quantize_per_token_bf16(const uint16_t* x, int64_t M, int64_t K, uint8_t* q,
                                          float* s, hipStream_t stream);
dg_status launch_quantize_per_block(const float* x, int64_t N, int64_t K, uint8_t* q, float* s,
                                     hipStream_t stream);
// Power-of-two scales: s holds E8M0 bytes, rows of K/128 padded to a multiple of 4.
dg_status launch_quantize_per_token_e8m0(const float* x, int64_t M, int64_t K, uint8_t* q,
                                          uint8_t* s, hipStream_t stream);
dg_status launch_quantize_per_block_e8m0(const float* x, int64_t N, int64_t K, uint8_t* q,
                                          uint8_t* s, hipStream_t stream);

}  // namespace dg
