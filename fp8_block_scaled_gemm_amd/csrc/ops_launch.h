// Internal launchers behind include/dg_ops.h (not exported), with the same
// contract as those of launch.h: sizes and pointers have been validated, a
// launcher only enqueues on `stream`.
#pragma once

#include "dg_ops.h"
#include "launch.h"

namespace dg {

struct TopkArgs {
    const void* logits;
    const float* bias;  // or null
    int32_t* ids;
    float* weights;
    int64_t T;
    int E, k, n_group, topk_group;
    bool sigmoid, renormalize;
    float scale;
};
dg_status launch_topk(const TopkArgs& a, bool bf16, hipStream_t stream);

struct TopkBackwardArgs {
    const void* logits;
    const int32_t* ids;
    const float* grad_weights;
    void* grad_logits;
    int64_t T;
    int E, k;
    bool sigmoid, renormalize;
    float scale;
};
dg_status launch_topk_backward(const TopkBackwardArgs& a, bool bf16, hipStream_t stream);

struct MoeArgs {
    const uint8_t* x;
    const void* sx;  // fp32, or E8M0 bytes with e8m0
    const int32_t* ids;
    const float* weights;
    const uint8_t* w13;
    const void* s13;
    const uint8_t* w2;
    const void* s2;
    uint16_t* y;
    int T, k, E, H, I;
    void* workspace;
};
int64_t moe_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I);
dg_status launch_moe(const MoeArgs& a, bool e8m0, hipStream_t stream);

struct LoraArgs {
    const uint8_t* A;
    const void* sa;
    const uint8_t* B;
    const void* sb;
    uint16_t* D;
    const uint16_t *x, *lora_a, *lora_b;
    const int32_t* ids;
    const float* scaling;
    int64_t M, N, K;
    int L, R;
    void* workspace;
};
int64_t lora_workspace(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R);
// DG_ERR_SHAPE where a launch of these sizes is past what a grid holds.
dg_status lora_limits(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R);
dg_status launch_lora(const LoraArgs& a, bool e8m0, hipStream_t stream);

}  // namespace dg
