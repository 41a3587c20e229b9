// The arithmetic of the quantizers, shared with the kernels that quantize on
// the way: correctly rounded x / scale and the power-of-two exponent.
#pragma once

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

}  // namespace dg
