// Device helpers shared by the gfx950 kernels of this library: vector types
// for MFMA operands and 16-byte accesses, direct loads to LDS with their
// waits, the FP8 matrix instruction and the e4m3 conversion.
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

typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<size_t>((lds_ptr_t)p));
}

// Raw buffer resource (gfx9 V#): `bytes` readable from `base`, stride 0.
// Loads at offsets past `bytes` return zero and touch no memory.
__device__ __forceinline__ v4u buffer_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    v4u r;
    r[0] = (uint32_t)a;
    r[1] = (uint32_t)(a >> 32) & 0xffffu;
    r[2] = bytes;
    r[3] = 0x00020000u;
    return r;
}

// One wave-wide direct load: lane l's bytes at buffer offset `off` land at
// dst + size*l in LDS (dst is wave-uniform, passed in M0).  Written as inline
// assembly on purpose: the compiler then does not track these LDS writes and
// cannot put a wait for the stage being filled in front of reads of the
// other stage (its alias tracking for such loads depends on control flow).
// The kernel orders them itself: every LDS read of a buffer is separated
// from the loads that refill it by a barrier (a compiler memory barrier as
// well), and a buffer is read only after the explicit vmcnt wait and barrier
// that publish it.  So the statements carry no memory clobber, and the
// compiler may still schedule unrelated LDS reads and arithmetic across them.
__device__ __forceinline__ void load_lds_16(const v4u& rsrc, uint32_t off, void* dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds_addr(dst)), "v"(off), "s"(rsrc) : "m0");
}
__device__ __forceinline__ void load_lds_4(const v4u& rsrc, uint32_t off, void* dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :: "s"(lds_addr(dst)), "v"(off), "s"(rsrc) : "m0");
}

// s_waitcnt on the vector-memory counter only (gfx9 encoding: vmcnt bits
// [3:0] and [15:14], expcnt and lgkmcnt left at their no-wait maxima).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// The same with lgkmcnt = 0: every LDS access this wave issued has completed.
template <int N>
__device__ __forceinline__ void wait_vmcnt_lgkm0() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}

// Workgroup barrier that is also a compiler barrier for memory accesses, but
// (unlike __syncthreads) waits for nothing: the kernel has already waited for
// exactly the loads the barrier publishes.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
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
