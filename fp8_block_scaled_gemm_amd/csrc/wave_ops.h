// Operations across the 64 lanes of a wave.
#pragma once

#include "device_common.h"

namespace dg {

// LDS written by some lanes of a wave before this is read by others after it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One register move across lanes (DPP), `none` where no lane feeds this one.
template <int kCtrl, int kRows, class T>
__device__ __forceinline__ T dpp_move(T v, T none) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),
                                                               __builtin_bit_cast(int, v), kCtrl, kRows, 0xf, false));
    } else {
        const v2u n = __builtin_bit_cast(v2u, none), x = __builtin_bit_cast(v2u, v);
        v2u r;
        r[0] = (uint32_t)__builtin_amdgcn_update_dpp((int)n[0], (int)x[0], kCtrl, kRows, 0xf, false);
        r[1] = (uint32_t)__builtin_amdgcn_update_dpp((int)n[1], (int)x[1], kCtrl, kRows, 0xf, false);
        return __builtin_bit_cast(T, r);
    }
}

// f over the wave's 64 values, in every lane (uniform); `none` is f's neutral
// value.  Six register moves across lanes; a shuffle through LDS takes about
// ten times as long as one.
template <class T, class F>
__device__ __forceinline__ T wave_reduce(T v, T none, F f) {
    v = f(v, dpp_move<0x111, 0xf>(v, none));  // within rows of 16: from 1, 2, 4, 8 lanes below
    v = f(v, dpp_move<0x112, 0xf>(v, none));
    v = f(v, dpp_move<0x114, 0xf>(v, none));
    v = f(v, dpp_move<0x118, 0xf>(v, none));
    v = f(v, dpp_move<0x142, 0xa>(v, none));  // row sums 0 -> 1, 2 -> 3
    v = f(v, dpp_move<0x143, 0xc>(v, none));  // rows 0-1 -> 2, 3
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
    } else {
        const v2u x = __builtin_bit_cast(v2u, v);
        return __builtin_bit_cast(T, v2u{(uint32_t)__builtin_amdgcn_readlane((int)x[0], 63),
                                         (uint32_t)__builtin_amdgcn_readlane((int)x[1], 63)});
    }
}

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
    return wave_reduce(v, (T)0, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ int wave_min(int v) {
    return wave_reduce(v, 0x7fffffff, [](int a, int b) { return a < b ? a : b; });
}

// The largest of each 16 lanes' values, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, dpp_move<0xb1, 0xf>(v, 0u));   // swap neighbours
    v = max(v, dpp_move<0x4e, 0xf>(v, 0u));   // swap pairs
    v = max(v, dpp_move<0x141, 0xf>(v, 0u));  // mirror 8
    return max(v, dpp_move<0x140, 0xf>(v, 0u));
}

}  // namespace dg
