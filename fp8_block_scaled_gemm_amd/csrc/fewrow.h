// The inner product of a few activation rows with streamed FP8 weights, shared
// by the decode-sized operators: one wave multiplies up to 16 R rows of A by
// 16 C rows of B, K block by K block, straight from memory to registers.
//
// Every byte of B is used by one wave only, so staging it through LDS would
// buy nothing; what counts is how many bytes are in flight.  A wave therefore
// keeps a ring of K blocks loading ahead of the one it multiplies.  The rows
// of A are few and shared by every wave of the launch: they come from cache.
//
// Fragment layout (v_mfma_f32_16x16x128_f8f6f4, B first): lane (lr, lg) holds
// 16-byte chunks lg and lg + 4 of row lr's 128-byte K block, for A and for B,
// and of the product output row lr, columns 4 lg .. 4 lg + 3.
#pragma once

#include "device_common.h"

namespace dg {

// One K block's operands of a wave.
template <int R, int C, bool kE8>
struct Block {
    using Scale = typename std::conditional<kE8, int, float>::type;
    v4u a[R][2], b[C][2];
    Scale sa[R], sb[C];
};

__device__ __forceinline__ void load_chunks(const uint8_t* p, v4u (&v)[2]) {
    v[0] = *reinterpret_cast<const v4u*>(p);
    v[1] = *reinterpret_cast<const v4u*>(p + 64);
}

// Rows that are not there read as zero through a bounds-checked buffer load,
// which touches no memory for them: offset kNoRow is past every buffer here.
constexpr uint32_t kNoRow = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)(uint32_t)bytes,
                                             0x00020000);
}

__device__ __forceinline__ void load_chunks(__amdgpu_buffer_rsrc_t buf, uint32_t off, v4u (&v)[2]) {
    v[0] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(buf, off, 0, 0));
    v[1] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(buf, off + 64, 0, 0));
}

// The K block's codes of one fragment as bf16, which holds every e4m3 value,
// in the four 32-wide steps of the bf16 matrix instruction.
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
__device__ __forceinline__ void widen(const v4u (&v)[2], v8bf (&out)[4]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        v2bf p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            p[q] = q & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[s >> 1][2 * (s & 1) + (q >> 1)], 1.0f, true)
                         : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[s >> 1][2 * (s & 1) + (q >> 1)], 1.0f, false);
        out[s] = v8bf{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
    }
}

// p * 2^(ea - 127) * 2^(eb - 127), E8M0 bytes (255 is NaN).
__device__ __forceinline__ float scale_e8(float p, int ea, int eb) {
    const float v = __builtin_amdgcn_ldexpf(p, ea + eb - 254);
    return ea == 255 || eb == 255 ? __builtin_nanf("") : v;
}

// The same as `multiply` below through the bf16 matrix instruction: its sums
// are exact to fp32 rounding, where the FP8 instruction aligns its 128
// products to about 16 bits (measured: 1.5e-5 against 1e-8 relative error of
// a K block).  For sums that are quantized next: an error there moves codes.
template <int R, int C, bool kE8>
__device__ __forceinline__ void multiply_exact(const Block<R, C, kE8>& k, int rows, v4f (&acc)[R][C]) {
    v8bf b[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c) widen(k.b[c], b[c]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r > 0 && 16 * r >= rows) break;
        v8bf a[4];
        widen(k.a[r], a);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 4; ++s) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[c][s], a[s], p, 0, 0, 0);
            if constexpr (kE8) {
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[r][c][q] += scale_e8(p[q], k.sa[r], k.sb[c]);
            } else {
                acc[r][c] += (k.sa[r] * k.sb[c]) * p;
            }
        }
    }
}

// acc += this block's scaled product; `rows` (uniform) of the 16 R rows count.
template <int R, int C, bool kE8>
__device__ __forceinline__ void multiply(const Block<R, C, kE8>& k, int rows, v4f (&acc)[R][C]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r > 0 && 16 * r >= rows) break;
        const v8i a = join(k.a[r][0], k.a[r][1]);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const v8i b = join(k.b[c][0], k.b[c][1]);
            if constexpr (kE8)
                acc[r][c] = mfma_block_e8(b, a, acc[r][c], k.sb[c], k.sa[r]);
            else
                acc[r][c] += (k.sa[r] * k.sb[c]) * mfma_block(b, a);
        }
    }
}

template <int R, int C>
__device__ __forceinline__ void clear(v4f (&acc)[R][C]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = v4f{0.f, 0.f, 0.f, 0.f};
}

// Scales per row of `kb` K blocks: fp32 as they are, E8M0 bytes padded to four.
template <bool kE8>
__host__ __device__ __forceinline__ int scale_pitch(int kb) {
    return kE8 ? (kb + 3) & ~3 : kb;
}

}  // namespace dg
