// The arithmetic of the quantizers, shared with the kernels that quantize on
// the way: correctly rounded x / scale and the power-of-two exponent.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace dg {

// x / b rounded to nearest even, given y = RN(1/b) finite and normal: q =
// RN(x y) is within an ulp of x/b, the remainder x - b q is exact (one FMA),
// and RN(q + (x - b q) y) is the correctly rounded quotient (Markstein's
// correction step).  Three operations instead of a full IEEE division.
__device__ __forceinline__ float quotient_rn(float x, float b, float y) {
    const float q0 = x * y;
    return __builtin_fmaf(__builtin_fmaf(-q0, b, x), y, q0);
}

// The power-of-two exponent of a block: amax = 1.f * 2^u needs e = u - 8
// when 1.f <= 1.75 (448 = 1.75 * 2^8, fraction bits 0x600000) and u - 7
// otherwise; zero and fp32 subnormals (below 2^-126, far below 448 * 2^-127)
// take the least exponent, -127.
__device__ __forceinline__ int e8m0_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int E = (int)(b >> 23);  // biased exponent; amax >= 0
    if (E == 0) return -127;
    return max(E - 135 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0), -127);
}

// 2^-e as an fp32 bit pattern (a normal number for e in [-127, 126]).
__device__ __forceinline__ float exp2_neg(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// Codes of four hidden values in a block whose largest magnitude has the bits
// `top` (a NaN's are the largest), and the block's scale or exponent byte: the
// per-token quantizer's recipe, with a NaN scale for a block that is not finite.
template <bool kE8>
__device__ __forceinline__ typename std::conditional<kE8, int, float>::type quantize_hidden(
    uint32_t top, const v4f& v, uint32_t& codes) {
    const float a = __uint_as_float(top);
    const bool finite = top < 0x7f800000u;
    float d[4];
    if constexpr (kE8) {
        const int ex = e8m0_exponent(a);
        const float y = exp2_neg(finite ? ex : 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) d[q] = v[q] * y;
        codes = e4m3x4_hw(d[0], d[1], d[2], d[3]);
        return finite ? ex + 127 : 255;
    } else {
        const float scale = a / 448.0f, y = 1.0f / scale;
        const bool fast = scale >= 1.17549435e-38f && y <= 3.40282347e38f;
        if (fast) {
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = quotient_rn(v[q], scale, y);
        } else {  // a scale below the normal range; a branch, not four divisions everywhere
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = v[q] / scale;
        }
        codes = top != 0 ? e4m3x4_hw(d[0], d[1], d[2], d[3]) : 0u;
        return finite ? scale : __builtin_nanf("");
    }
}

}  // namespace dg
