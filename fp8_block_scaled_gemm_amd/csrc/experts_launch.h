// Internal launchers behind include/dg_experts.h and include/dg_int8.h (not
// exported), with the same contract as those of launch.h: sizes and pointers
// have been validated, a launcher only enqueues on `stream`.
#pragma once

#include "dg_experts.h"
#include "dg_int8.h"
#include "launch.h"

namespace dg {

// How a row of activations is held: bf16, codes with a scale per 128 columns
// (fp32, or an E8M0 byte), or int8 with one fp32 scale.
enum class Held : int { Bf16 = 0, Fp8 = 1, Fp8E8 = 2, Int8 = 3 };

struct SortArgs {
    const int32_t* ids;
    int32_t *rows, *layout, *offsets;
    int64_t T, M;
    int k, E;
    void* workspace;
};
int64_t sort_workspace(int64_t T, int64_t k, int64_t E);
dg_status launch_sort(const SortArgs& a, hipStream_t stream);

struct DispatchArgs {
    SortArgs sort;
    const uint16_t* x;
    void* out;  // bf16 bits, or codes
    void* s;    // scales, null for Bf16
    int64_t H;
};
// DG_ERR_SHAPE where a launch of these sizes is past what a grid holds.
dg_status dispatch_limits(int64_t T, int64_t k, int64_t E, int64_t H, int64_t M, Held held);
dg_status launch_dispatch(const DispatchArgs& a, Held held, hipStream_t stream);

struct UnpermuteArgs {
    const uint16_t* y;
    const int32_t* rows;
    const float* weights;  // or null
    uint16_t* out;
    int64_t T, H, M;
    int k;
};
dg_status launch_unpermute(const UnpermuteArgs& a, hipStream_t stream);

struct UnpermuteBackwardArgs {
    const uint16_t *grad, *y;
    const int32_t* rows;
    const float* weights;   // or null
    const int32_t* layout;  // or null
    uint16_t* grad_y;       // or null
    float* grad_weights;    // or null
    int64_t T, H, M;
    int k;
};
dg_status launch_unpermute_backward(const UnpermuteBackwardArgs& a, hipStream_t stream);

struct SwigluArgs {
    const uint16_t* z;
    const int32_t* layout;  // or null
    void* out;
    void* s;
    int64_t M, I;
};
dg_status launch_swiglu(const SwigluArgs& a, Held held, hipStream_t stream);

struct SwigluBackwardArgs {
    const uint16_t *z, *grad_h;
    const int32_t* layout;  // or null
    uint16_t* grad_z;
    int64_t M, I;
};
dg_status launch_swiglu_backward(const SwigluBackwardArgs& a, hipStream_t stream);

struct Int8Args {
    const int8_t* A;
    const float* sa;
    const int8_t* B;
    const float* sb;
    uint16_t* D;
    const int32_t* layout;  // null for the dense form
    int64_t rows, N, K, G;
};
dg_status launch_int8_gemm(const Int8Args& a, hipStream_t stream);
dg_status launch_quantize_int8(const void* x, bool bf16, int64_t M, int64_t K, int8_t* q, float* s,
                               hipStream_t stream);

}  // namespace dg
