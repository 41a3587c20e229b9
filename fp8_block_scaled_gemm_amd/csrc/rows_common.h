// Rows of bf16 activations in registers, and the int8 recipe of a row, shared
// by the kernels that quantize rows on the way.
#pragma once

#include "quantize_common.h"
#include "wave_ops.h"

namespace dg {

// Eight bf16 in four words, the lower half of a word first, and back, rounded
// to nearest even.  A bf16 is the upper half of its fp32.
__device__ __forceinline__ void unpack_bf16(const v4u& raw, float (&f)[8]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        f[2 * w] = __uint_as_float(raw[w] << 16);
        f[2 * w + 1] = __uint_as_float(raw[w] & 0xffff0000u);
    }
}
__device__ __forceinline__ v4u pack_bf16(const float (&f)[8]) {
    v4u r;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        r[w] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{f[2 * w], f[2 * w + 1]}), v2bf));
    return r;
}

__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of an int8 row whose largest magnitude has the bits `top` (a NaN's
// are the largest), and its codes, four to a word.
struct Int8Row {
    float scale, inverse;
    bool fast, zero;
    __device__ __forceinline__ explicit Int8Row(uint32_t top) {
        scale = __uint_as_float(top) / 127.0f;
        inverse = 1.0f / scale;
        fast = scale >= 1.17549435e-38f && inverse <= 3.40282347e38f;
        zero = scale == 0.0f || top >= 0x7f800000u;
        if (top >= 0x7f800000u) scale = __builtin_nanf("");
    }
    // The code in the lowest byte: the correctly rounded quotient, then the nearest
    // integer, ties to even, as the lowest bits of its sum with 1.5 * 2^23.  A scale
    // below the normal range is coarse, and a quotient may pass 127.
    __device__ __forceinline__ uint32_t code(float v) const {
        const float d = fast ? quotient_rn(v, scale, inverse) : v / scale;
        return __float_as_uint(__builtin_amdgcn_fmed3f(d, -127.0f, 127.0f) + 12582912.0f);
    }
    __device__ __forceinline__ v2u codes(const float (&f)[8]) const {
        v2u r;
#pragma unroll
        for (int w = 0; w < 2; ++w) {  // v_perm_b32: bytes 0-3 are the second operand's, 4-7 the first's
            const uint32_t lo = __builtin_amdgcn_perm(code(f[4 * w + 1]), code(f[4 * w]), 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(code(f[4 * w + 3]), code(f[4 * w + 2]), 0x0c0c0400u);
            r[w] = zero ? 0u : __builtin_amdgcn_perm(hi, lo, 0x05040100u);
        }
        return r;
    }
};

// One row of `width` times 8 columns into int8, by G threads of which this is
// the `id`-th: all of a workgroup's 256, or a wave's 64.  `load` gives the fp32
// values of 8 columns, `store` takes their codes.  Each thread keeps C loads; a
// row that is wider than G C (C = 0: any) is loaded twice, the second time from
// the cache.  Returns the row's scale.
template <int G, int C, class Load, class Store>
__device__ __forceinline__ float int8_row(int64_t width, int id, uint32_t* lds, Load load, Store store) {
    static_assert(G == 64 || G == 256, "a wave or a workgroup");
    float f[C > 0 ? C : 1][8];
    uint32_t top = 0;
    auto look = [&](const float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, magnitude_bits(v[e]));
    };
    if constexpr (C > 0) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (id + i * G < width) load((int64_t)(id + i * G), f[i]);
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (id + i * G < width) look(f[i]);
    } else {
        for (int64_t c = id; c < width; c += G) {
            load(c, f[0]);
            look(f[0]);
        }
    }
    top = wave_max(top);
    if constexpr (G == 256) {
        if ((id & 63) == 0) lds[id >> 6] = top;
        __syncthreads();
        top = max(max(lds[0], lds[1]), max(lds[2], lds[3]));
    }
    const Int8Row row(top);
    if constexpr (C > 0) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (id + i * G < width) store((int64_t)(id + i * G), row.codes(f[i]));
    } else {
        for (int64_t c = id; c < width; c += G) {
            load(c, f[0]);
            store(c, row.codes(f[0]));
        }
    }
    return row.scale;
}

// Codes of a 128-column block that eight lanes hold, lane l its columns 8l ..
// 8l+7 and 64+8l .. 64+8l+7: the block's scale (kE8: exponent byte, in every
// lane) and, in `line` (LDS, the group's own 128 bytes), the codes in order.
// The lanes are in one wave, whose LDS accesses are ordered: no barrier.
template <bool kE8>
__device__ __forceinline__ auto block_codes(const float (&f)[2][8], uint8_t* line, int lane) {
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, magnitude_bits(f[h][e]));
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 8));
    typename std::conditional<kE8, int, float>::type scale;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t lo, hi;
        scale = quantize_hidden<kE8>(top, v4f{f[h][0], f[h][1], f[h][2], f[h][3]}, lo);
        quantize_hidden<kE8>(top, v4f{f[h][4], f[h][5], f[h][6], f[h][7]}, hi);
        *reinterpret_cast<v2u*>(line + 64 * h + 8 * lane) = v2u{lo, hi};
    }
    wave_sync();
    return scale;
}

}  // namespace dg
