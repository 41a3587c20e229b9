// The C ABI of include/dg_experts.h and include/dg_int8.h: host-side argument
// checks, then the enqueue.  Nothing here touches the GPU before every check
// has passed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "experts_launch.h"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 62;
constexpr int64_t kMaxRows = 0x7fffffff;

bool product_ok(int64_t a, int64_t b) { return a == 0 || b <= kMaxElems / a; }

dg_status check_ptrs(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (p == nullptr) return DG_ERR_NULL;
    for (const void* p : ptrs)
        if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return DG_ERR_ALIGN;
    return DG_OK;
}

// Pointers that may be null.
dg_status check_given(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (p != nullptr && check_ptrs({p}) != DG_OK) return DG_ERR_ALIGN;
    return DG_OK;
}

hipStream_t on(void* stream) { return static_cast<hipStream_t>(stream); }

dg_status check_sort(int64_t T, int64_t k, int64_t E) {
    if (T < 0 || k < 1 || k > 64 || E < 1 || E > 4096 || T > (int64_t(1) << 30) / k) return DG_ERR_SHAPE;
    return DG_OK;
}

int64_t sort_rows(int64_t T, int64_t k, int64_t E) {
    const int64_t P = T * k;
    return (P + 127 * std::min(E, P)) / 128 * 128;
}

// Of the sort that every dispatch call starts with.
dg_status check_plan(const int32_t* ids, const int32_t* rows, const int32_t* layout, const int32_t* offsets, int64_t T,
                     int64_t k, int64_t E, int64_t M, const void* workspace, int64_t workspace_bytes, bool pointers) {
    if (!pointers) {
        const dg_status s = check_sort(T, k, E);
        if (s != DG_OK) return s;
        if (M < sort_rows(T, k, E) || M % 128 != 0 || M > kMaxRows) return DG_ERR_SHAPE;
        return workspace_bytes < dg::sort_workspace(T, k, E) ? DG_ERR_SHAPE : DG_OK;
    }
    dg_status s = check_ptrs({offsets});
    if (s == DG_OK && T > 0) s = check_ptrs({ids, rows});
    if (s == DG_OK && M > 0) s = check_ptrs({layout});
    if (s == DG_OK && dg::sort_workspace(T, k, E) > 0) s = check_ptrs({workspace});
    return s;
}

dg_status dispatch(const uint16_t* x, const int32_t* ids, void* out, void* scales, int32_t* rows, int32_t* layout,
                   int32_t* offsets, int64_t T, int64_t k, int64_t E, int64_t H, int64_t M, void* workspace,
                   int64_t workspace_bytes, void* stream, dg::Held held) {
    dg_status s = check_plan(ids, rows, layout, offsets, T, k, E, M, workspace, workspace_bytes, false);
    if (s != DG_OK) return s;
    const int64_t unit = held == dg::Held::Bf16 ? 8 : 128;
    if (H <= 0 || H % unit != 0 || H >= (int64_t(1) << 24)) return DG_ERR_SHAPE;
    if ((s = dg::dispatch_limits(T, k, E, H, M, held)) != DG_OK) return s;
    s = check_plan(ids, rows, layout, offsets, T, k, E, M, workspace, workspace_bytes, true);
    if (s == DG_OK && T > 0) s = check_ptrs({x});
    if (s == DG_OK && M > 0) s = held == dg::Held::Bf16 ? check_ptrs({out}) : check_ptrs({out, scales});
    if (s != DG_OK) return s;
    const dg::DispatchArgs a{{ids, rows, layout, offsets, T, M, (int)k, (int)E, workspace}, x, out, scales, H};
    return dg::launch_dispatch(a, held, on(stream));
}

dg_status check_rows(int64_t T, int64_t k, int64_t H, int64_t M) {
    if (T < 0 || T > kMaxRows || M < 0 || M > kMaxRows || k < 1 || k > 64) return DG_ERR_SHAPE;
    return H <= 0 || H % 8 != 0 || H >= (int64_t(1) << 24) ? DG_ERR_SHAPE : DG_OK;
}

dg_status swiglu(const uint16_t* z, const int32_t* layout, void* out, void* scales, int64_t M, int64_t I, void* stream,
                 dg::Held held) {
    const int64_t unit = held == dg::Held::Bf16 ? 8 : 128;
    if (M < 0 || M > kMaxRows || I <= 0 || I % unit != 0 || I >= (int64_t(1) << 23)) return DG_ERR_SHAPE;
    if (M == 0) return DG_OK;
    dg_status s = held == dg::Held::Bf16 ? check_ptrs({z, out}) : check_ptrs({z, out, scales});
    if (s == DG_OK) s = check_given({layout});
    if (s != DG_OK) return s;
    return dg::launch_swiglu(dg::SwigluArgs{z, layout, out, scales, M, I}, held, on(stream));
}

dg_status int8_gemm(const int8_t* A, const float* sa, const int8_t* B, const float* sb, uint16_t* D,
                    const int32_t* layout, int64_t rows, int64_t N, int64_t K, int64_t G, void* stream, bool grouped) {
    if (N <= 0 || N % 8 != 0 || N > kMaxRows || K <= 0 || K % 128 != 0 || K >= (1 << 17)) return DG_ERR_SHAPE;
    if (G < 1 || G > kMaxRows || !product_ok(G, N * K)) return DG_ERR_SHAPE;
    if (rows < 0 || rows > kMaxRows || (grouped && rows % 128 != 0)) return DG_ERR_SHAPE;
    if (rows == 0) return DG_OK;
    dg_status s = check_ptrs({A, sa, B, sb, D});
    if (s == DG_OK && grouped) s = check_ptrs({layout});
    if (s != DG_OK) return s;
    return dg::launch_int8_gemm(dg::Int8Args{A, sa, B, sb, D, grouped ? layout : nullptr, rows, N, K, G}, on(stream));
}

dg_status quantize_int8(const void* x, bool bf16, int64_t M, int64_t K, int8_t* q, float* s, void* stream) {
    if (M < 0 || K <= 0 || K % 128 != 0 || K >= (int64_t(1) << 24) || !product_ok(M, K)) return DG_ERR_SHAPE;
    if (M == 0) return DG_OK;
    const dg_status st = check_ptrs({x, q, s});
    if (st != DG_OK) return st;
    return dg::launch_quantize_int8(x, bf16, M, K, q, s, on(stream));
}

}  // namespace

extern "C" {

dg_status dg_moe_sort(const int32_t* ids, int32_t* rows, int32_t* layout, int32_t* offsets, int64_t T, int64_t k,
                      int64_t E, int64_t M, void* workspace, int64_t workspace_bytes, void* stream) {
    dg_status s = check_plan(ids, rows, layout, offsets, T, k, E, M, workspace, workspace_bytes, false);
    if (s == DG_OK) s = check_plan(ids, rows, layout, offsets, T, k, E, M, workspace, workspace_bytes, true);
    if (s != DG_OK) return s;
    return dg::launch_sort(dg::SortArgs{ids, rows, layout, offsets, T, M, (int)k, (int)E, workspace}, on(stream));
}

dg_status dg_moe_sort_rows(int64_t T, int64_t k, int64_t E, int64_t* rows) {
    const dg_status s = check_sort(T, k, E);
    if (s != DG_OK) return s;
    if (sort_rows(T, k, E) > kMaxRows) return DG_ERR_SHAPE;
    if (rows == nullptr) return DG_ERR_NULL;
    *rows = sort_rows(T, k, E);
    return DG_OK;
}

dg_status dg_moe_sort_workspace(int64_t T, int64_t k, int64_t E, int64_t* bytes) {
    const dg_status s = check_sort(T, k, E);
    if (s != DG_OK) return s;
    if (bytes == nullptr) return DG_ERR_NULL;
    *bytes = dg::sort_workspace(T, k, E);
    return DG_OK;
}

dg_status dg_moe_dispatch(const uint16_t* x, const int32_t* ids, uint16_t* out, int32_t* rows, int32_t* layout,
                          int32_t* offsets, int64_t T, int64_t k, int64_t E, int64_t H, int64_t M, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    return dispatch(x, ids, out, nullptr, rows, layout, offsets, T, k, E, H, M, workspace, workspace_bytes, stream,
                    dg::Held::Bf16);
}

dg_status dg_moe_dispatch_fp8(const uint16_t* x, const int32_t* ids, uint8_t* q, float* s, int32_t* rows,
                              int32_t* layout, int32_t* offsets, int64_t T, int64_t k, int64_t E, int64_t H, int64_t M,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    return dispatch(x, ids, q, s, rows, layout, offsets, T, k, E, H, M, workspace, workspace_bytes, stream,
                    dg::Held::Fp8);
}

dg_status dg_moe_dispatch_fp8_e8m0(const uint16_t* x, const int32_t* ids, uint8_t* q, uint8_t* s, int32_t* rows,
                                   int32_t* layout, int32_t* offsets, int64_t T, int64_t k, int64_t E, int64_t H,
                                   int64_t M, void* workspace, int64_t workspace_bytes, void* stream) {
    return dispatch(x, ids, q, s, rows, layout, offsets, T, k, E, H, M, workspace, workspace_bytes, stream,
                    dg::Held::Fp8E8);
}

dg_status dg_moe_dispatch_int8(const uint16_t* x, const int32_t* ids, int8_t* q, float* s, int32_t* rows,
                               int32_t* layout, int32_t* offsets, int64_t T, int64_t k, int64_t E, int64_t H, int64_t M,
                               void* workspace, int64_t workspace_bytes, void* stream) {
    return dispatch(x, ids, q, s, rows, layout, offsets, T, k, E, H, M, workspace, workspace_bytes, stream,
                    dg::Held::Int8);
}

dg_status dg_moe_unpermute(const uint16_t* y, const int32_t* rows, const float* weights, uint16_t* out, int64_t T,
                           int64_t k, int64_t H, int64_t M, void* stream) {
    dg_status s = check_rows(T, k, H, M);
    if (s != DG_OK || T == 0) return s;
    s = check_ptrs({rows, out});
    if (s == DG_OK && M > 0) s = check_ptrs({y});
    if (s == DG_OK) s = check_given({weights});
    if (s != DG_OK) return s;
    return dg::launch_unpermute(dg::UnpermuteArgs{y, rows, weights, out, T, H, M, (int)k}, on(stream));
}

dg_status dg_moe_unpermute_backward(const uint16_t* grad, const uint16_t* y, const int32_t* rows, const float* weights,
                                    const int32_t* layout, uint16_t* grad_y, float* grad_weights, int64_t T, int64_t k,
                                    int64_t H, int64_t M, void* stream) {
    dg_status s = check_rows(T, k, H, M);
    if (s != DG_OK || (T == 0 && M == 0)) return s;
    if (grad_y == nullptr && grad_weights == nullptr && M > 0 && T > 0) return DG_ERR_NULL;
    if (T > 0) s = check_ptrs({grad, rows});
    if (s == DG_OK && T > 0 && M > 0 && grad_weights != nullptr) s = check_ptrs({y});
    if (s == DG_OK) s = check_given({weights, layout, grad_y, grad_weights});
    if (s != DG_OK) return s;
    return dg::launch_unpermute_backward(
        dg::UnpermuteBackwardArgs{grad, y, rows, weights, layout, grad_y, grad_weights, T, H, M, (int)k}, on(stream));
}

dg_status dg_swiglu(const uint16_t* z, const int32_t* layout, uint16_t* h, int64_t M, int64_t I, void* stream) {
    return swiglu(z, layout, h, nullptr, M, I, stream, dg::Held::Bf16);
}

dg_status dg_swiglu_quantize_fp8(const uint16_t* z, const int32_t* layout, uint8_t* q, float* s, int64_t M, int64_t I,
                                 void* stream) {
    return swiglu(z, layout, q, s, M, I, stream, dg::Held::Fp8);
}

dg_status dg_swiglu_quantize_fp8_e8m0(const uint16_t* z, const int32_t* layout, uint8_t* q, uint8_t* s, int64_t M,
                                      int64_t I, void* stream) {
    return swiglu(z, layout, q, s, M, I, stream, dg::Held::Fp8E8);
}

dg_status dg_swiglu_quantize_int8(const uint16_t* z, const int32_t* layout, int8_t* q, float* s, int64_t M, int64_t I,
                                  void* stream) {
    return swiglu(z, layout, q, s, M, I, stream, dg::Held::Int8);
}

dg_status dg_swiglu_backward(const uint16_t* z, const uint16_t* grad_h, const int32_t* layout, uint16_t* grad_z,
                             int64_t M, int64_t I, void* stream) {
    if (M < 0 || M > kMaxRows || I <= 0 || I % 8 != 0 || I >= (int64_t(1) << 23)) return DG_ERR_SHAPE;
    if (M == 0) return DG_OK;
    dg_status s = check_ptrs({z, grad_h, grad_z});
    if (s == DG_OK) s = check_given({layout});
    if (s != DG_OK) return s;
    return dg::launch_swiglu_backward(dg::SwigluBackwardArgs{z, grad_h, layout, grad_z, M, I}, on(stream));
}

dg_status dg_int8_gemm_nt(const int8_t* A, const float* sa, const int8_t* B, const float* sb, uint16_t* D, int64_t M,
                          int64_t N, int64_t K, void* stream) {
    return int8_gemm(A, sa, B, sb, D, nullptr, M, N, K, 1, stream, false);
}

dg_status dg_int8_gemm_grouped_contiguous(const int8_t* A, const float* sa, const int8_t* B, const float* sb,
                                          uint16_t* D, const int32_t* grouped_layout, int64_t M_sum, int64_t N,
                                          int64_t K, int64_t G, void* stream) {
    return int8_gemm(A, sa, B, sb, D, grouped_layout, M_sum, N, K, G, stream, true);
}

dg_status dg_quantize_int8_per_row(const float* x, int64_t M, int64_t K, int8_t* q, float* s, void* stream) {
    return quantize_int8(x, false, M, K, q, s, stream);
}

dg_status dg_quantize_int8_per_row_bf16(const uint16_t* x, int64_t M, int64_t K, int8_t* q, float* s, void* stream) {
    return quantize_int8(x, true, M, K, q, s, stream);
}

}  // extern "C"
