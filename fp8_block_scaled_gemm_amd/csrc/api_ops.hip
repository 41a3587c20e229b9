// The C ABI of include/dg_ops.h: host-side argument checks, then the enqueue.
// Nothing here touches the GPU before every check has passed.
#include "dg_ops.h"

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "ops_launch.h"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 62;

bool product_ok(int64_t a, int64_t b) { return a == 0 || b <= kMaxElems / a; }

dg_status check_ptrs(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (p == nullptr) return DG_ERR_NULL;
    for (const void* p : ptrs)
        if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return DG_ERR_ALIGN;
    return DG_OK;
}

bool scoring_ok(int scoring) { return scoring == DG_SCORE_SOFTMAX || scoring == DG_SCORE_SIGMOID; }

dg_status topk(const void* logits, const float* bias, int32_t* ids, float* weights, int64_t T,
               int64_t E, int64_t k, int64_t n_group, int64_t topk_group, int scoring,
               int renormalize, float scale, void* stream, bool bf16) {
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 64 || !product_ok(T, E * 4)) return DG_ERR_SHAPE;
    if (n_group < 1 || n_group > 64 || E % n_group != 0) return DG_ERR_SHAPE;
    if (topk_group < 1 || topk_group > n_group || k > topk_group * (E / n_group)) return DG_ERR_SHAPE;
    if (!scoring_ok(scoring)) return DG_ERR_UNSUPPORTED;
    if (T == 0) return DG_OK;
    dg_status s = check_ptrs({logits, ids, weights});
    if (s == DG_OK && bias != nullptr) s = check_ptrs({bias});
    if (s != DG_OK) return s;
    const dg::TopkArgs a{logits, bias, ids, weights, T, (int)E, (int)k, (int)n_group, (int)topk_group,
                         scoring == DG_SCORE_SIGMOID, renormalize != 0, scale};
    return dg::launch_topk(a, bf16, static_cast<hipStream_t>(stream));
}

dg_status topk_backward(const void* logits, const int32_t* ids, const float* grad_weights,
                        void* grad_logits, int64_t T, int64_t E, int64_t k, int scoring,
                        int renormalize, float scale, void* stream, bool bf16) {
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 64 || !product_ok(T, E * 4)) return DG_ERR_SHAPE;
    if (!scoring_ok(scoring)) return DG_ERR_UNSUPPORTED;
    if (T == 0) return DG_OK;
    const dg_status s = check_ptrs({logits, ids, grad_weights, grad_logits});
    if (s != DG_OK) return s;
    const dg::TopkBackwardArgs a{logits, ids, grad_weights, grad_logits, T, (int)E, (int)k,
                                 scoring == DG_SCORE_SIGMOID, renormalize != 0, scale};
    return dg::launch_topk_backward(a, bf16, static_cast<hipStream_t>(stream));
}

dg_status check_moe(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
    if (T < 0 || T > 256 || k < 1 || k > 16 || E < 1 || E > 65536) return DG_ERR_SHAPE;
    if (H <= 0 || H % 128 != 0 || H > 16384 || I <= 0 || I % 128 != 0 || I > 16384) return DG_ERR_SHAPE;
    return DG_OK;
}

dg_status moe(const uint8_t* x, const void* sx, const int32_t* ids, const float* weights,
              const uint8_t* w13, const void* s13, const uint8_t* w2, const void* s2, uint16_t* y,
              int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, void* workspace,
              int64_t workspace_bytes, void* stream, bool e8) {
    dg_status s = check_moe(T, k, E, H, I);
    if (s != DG_OK) return s;
    if (T == 0) return DG_OK;
    if (workspace_bytes < dg::moe_workspace(T, k, E, H, I)) return DG_ERR_SHAPE;
    s = check_ptrs({x, sx, ids, weights, w13, s13, w2, s2, y, workspace});
    if (s != DG_OK) return s;
    const dg::MoeArgs a{x,  sx,     ids,    weights, w13,    s13,    w2, s2, y, (int)T,
                        (int)k, (int)E, (int)H,  (int)I, workspace};
    return dg::launch_moe(a, e8, static_cast<hipStream_t>(stream));
}

dg_status check_lora(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    if (N <= 0 || N % 8 != 0 || N >= (int64_t(1) << 22)) return DG_ERR_SHAPE;
    // an adapter's R <= 128 rows of K bf16 are addressed with 31-bit offsets
    if (K <= 0 || K % 128 != 0 || K >= (int64_t(1) << 23)) return DG_ERR_SHAPE;
    if (M < 0 || M > 0x7fffffffLL || L < 1 || L > 65536) return DG_ERR_SHAPE;
    if (R < 8 || R > 128 || R % 8 != 0) return DG_ERR_SHAPE;
    // refused here, as the dense launch would do so behind the adapters' own;
    // below these sizes no grid is too large, in the smallest tiles
    if (M > (1 << 24) || ((M + 127) / 128) * ((N + 31) / 32) > (1 << 23)) return dg::lora_limits(M, N, K, L, R);
    return DG_OK;
}

dg_status lora(const uint8_t* A, const void* sa, const uint8_t* B, const void* sb, uint16_t* D,
               const uint16_t* x, const uint16_t* lora_a, const uint16_t* lora_b, const int32_t* ids,
               const float* scaling, int64_t M, int64_t N, int64_t K, int64_t L, int64_t R,
               void* workspace, int64_t workspace_bytes, void* stream, bool e8) {
    dg_status s = check_lora(M, N, K, L, R);
    if (s != DG_OK) return s;
    if (M == 0) return DG_OK;
    if (workspace_bytes < dg::lora_workspace(M, N, K, L, R)) return DG_ERR_SHAPE;
    s = check_ptrs({A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, workspace});
    if (s != DG_OK) return s;
    const dg::LoraArgs a{A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, M, N, K, (int)L, (int)R,
                         workspace};
    return dg::launch_lora(a, e8, static_cast<hipStream_t>(stream));
}

}  // namespace

extern "C" {

dg_status dg_moe_topk(const float* logits, const float* bias, int32_t* ids, float* weights,
                      int64_t T, int64_t E, int64_t k, int64_t n_group, int64_t topk_group,
                      int scoring, int renormalize, float scale, void* stream) {
    return topk(logits, bias, ids, weights, T, E, k, n_group, topk_group, scoring, renormalize, scale,
                stream, false);
}

dg_status dg_moe_topk_bf16(const uint16_t* logits, const float* bias, int32_t* ids, float* weights,
                           int64_t T, int64_t E, int64_t k, int64_t n_group, int64_t topk_group,
                           int scoring, int renormalize, float scale, void* stream) {
    return topk(logits, bias, ids, weights, T, E, k, n_group, topk_group, scoring, renormalize, scale,
                stream, true);
}

dg_status dg_moe_topk_backward(const float* logits, const int32_t* ids, const float* grad_weights,
                               float* grad_logits, int64_t T, int64_t E, int64_t k, int scoring,
                               int renormalize, float scale, void* stream) {
    return topk_backward(logits, ids, grad_weights, grad_logits, T, E, k, scoring, renormalize, scale,
                         stream, false);
}

dg_status dg_moe_topk_backward_bf16(const uint16_t* logits, const int32_t* ids,
                                    const float* grad_weights, uint16_t* grad_logits, int64_t T,
                                    int64_t E, int64_t k, int scoring, int renormalize, float scale,
                                    void* stream) {
    return topk_backward(logits, ids, grad_weights, grad_logits, T, E, k, scoring, renormalize, scale,
                         stream, true);
}

dg_status dg_moe_mlp_fp8(const uint8_t* x, const float* sx, const int32_t* ids, const float* weights,
                         const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2,
                         uint16_t* y, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I,
                         void* workspace, int64_t workspace_bytes, void* stream) {
    return moe(x, sx, ids, weights, w13, s13, w2, s2, y, T, k, E, H, I, workspace, workspace_bytes,
               stream, false);
}

dg_status dg_moe_mlp_fp8_e8m0(const uint8_t* x, const uint8_t* sx, const int32_t* ids,
                              const float* weights, const uint8_t* w13, const uint8_t* s13,
                              const uint8_t* w2, const uint8_t* s2, uint16_t* y, int64_t T,
                              int64_t k, int64_t E, int64_t H, int64_t I, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    return moe(x, sx, ids, weights, w13, s13, w2, s2, y, T, k, E, H, I, workspace, workspace_bytes,
               stream, true);
}

dg_status dg_moe_mlp_fp8_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I,
                                   int64_t* bytes) {
    const dg_status s = check_moe(T, k, E, H, I);
    if (s != DG_OK) return s;
    if (bytes == nullptr) return DG_ERR_NULL;
    *bytes = dg::moe_workspace(T, k, E, H, I);
    return DG_OK;
}

dg_status dg_fp8_gemm_nt_lora(const uint8_t* A, const float* sa, const uint8_t* B, const float* sb,
                              uint16_t* D, const uint16_t* x, const uint16_t* lora_a,
                              const uint16_t* lora_b, const int32_t* ids, const float* scaling,
                              int64_t M, int64_t N, int64_t K, int64_t L, int64_t R,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    return lora(A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, M, N, K, L, R, workspace,
                workspace_bytes, stream, false);
}

dg_status dg_fp8_gemm_nt_lora_e8m0(const uint8_t* A, const uint8_t* sa, const uint8_t* B,
                                   const uint8_t* sb, uint16_t* D, const uint16_t* x,
                                   const uint16_t* lora_a, const uint16_t* lora_b,
                                   const int32_t* ids, const float* scaling, int64_t M, int64_t N,
                                   int64_t K, int64_t L, int64_t R, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    return lora(A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, M, N, K, L, R, workspace,
                workspace_bytes, stream, true);
}

dg_status dg_fp8_gemm_nt_lora_workspace(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R,
                                        int64_t* bytes) {
    const dg_status s = check_lora(M, N, K, L, R);
    if (s != DG_OK) return s;
    if (bytes == nullptr) return DG_ERR_NULL;
    *bytes = dg::lora_workspace(M, N, K, L, R);
    return DG_OK;
}

}  // extern "C"
