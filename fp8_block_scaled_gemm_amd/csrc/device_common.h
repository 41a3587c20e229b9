// Device helpers shared by the gfx950 kernels of this library: vector types
// for MFMA operands and 16-byte accesses, the FP8 matrix instruction and the
// e4m3 conversion.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));  // 16-byte global/LDS chunk
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// Four fp32 values -> four OCP E4M3FN codes (byte i = value i, sign kept)
// with the hardware conversion (v_cvt_pk_fp8_f32: round to nearest even,
// subnormal codes below 2^-6).  Inputs are clamped to +-448 first
// (v_med3_f32), so the conversion never sees a value past the largest finite
// e4m3: results saturate at +-448.
__device__ __forceinline__ uint32_t e4m3x4_hw(float a, float b, float c, float d) {
    const float lim = 448.0f;
    a = __builtin_amdgcn_fmed3f(a, -lim, lim);
    b = __builtin_amdgcn_fmed3f(b, -lim, lim);
    c = __builtin_amdgcn_fmed3f(c, -lim, lim);
    d = __builtin_amdgcn_fmed3f(d, -lim, lim);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}

// The partial product of one 128-wide K block of a 16x16 sub-tile.
__device__ __forceinline__ v4f mfma_block(const v8i& b, const v8i& a) {
    const v4f zero = {0.f, 0.f, 0.f, 0.f};
    // format 0 = e4m3 for both operands; zero scale operands select the
    // unscaled instruction
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, zero, 0, 0, 0, 0, 0, 0);
}

// acc + 2^(eb-127) * 2^(ea-127) * (B_blk A_blk^T) in one instruction.  Each
// lane passes one E8M0 byte per operand in bits 0-7 (opsel 0): operand 0's
// (eb) applies to B row (lane & 15) of the sub-tile, operand 1's (ea) to A
// row (lane & 15), each for the 32-wide K group (lane >> 4); a block's four
// groups share one scale, so every lane passes its row's block scale.
__device__ __forceinline__ v4f mfma_block_e8(const v8i& b, const v8i& a, const v4f& c, int eb,
                                              int ea) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, 0, eb, 0, ea);
}

__device__ __forceinline__ v8i join(const v4u& lo, const v4u& hi) {
    return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

}  // namespace dg
