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
