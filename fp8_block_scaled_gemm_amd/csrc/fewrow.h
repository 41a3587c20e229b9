// The product of a few activation rows with streamed FP8 weights, shared by
// the decode-sized operators: one wave multiplies up to 16 R rows of A by 16 C
// rows of B, K block by K block.  Every byte of B is used once, so what counts
// is how many bytes are in flight: rings in LDS, filled by direct loads, keep
// K blocks loading ahead of the one that is multiplied (see panels, below).
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

// Rows that are not there read as zero through a bounds-checked buffer load,
// which touches no memory for them: offset kNoRow is past every buffer here.
constexpr uint32_t kNoRow = 0x80000000u;

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
// a K block).  The expert layer's products take it: the first one's sums are
// quantized next, where an error moves codes, and the second one's are promised
// in 32 bits (two products that cancel would take the bits of the others with
// them).  It costs the widening, 16 conversions a fragment: the second product
// 0 to 5% of a call (one token of 8 experts of 7168 x 2048 68.4 -> 69.1 us, 64
// tokens of 16 146 -> 149.5, 251 tokens, one pair in eight here, 145.5 -> 146.0,
// 256 tokens of 16 experts of 4096 x 1024 160 -> 168.5).
template <int R, int C, bool kE8>
__device__ __forceinline__ void multiply_exact(const Block<R, C, kE8>& k, int rows, v4f (&acc)[R][C]) {
    v8bf b[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c) widen(k.b[c], b[c]);
    // Two row tiles at a time with two column tiles: four chains of dependent
    // products in flight.  With one column tile it is one, as most experts of a
    // spread batch have few rows (the 251 tokens above: 164 us in pairs).
    constexpr int kPair = R >= 2 && C >= 2 ? 2 : 1;
#pragma unroll
    for (int r0 = 0; r0 < R; r0 += kPair) {
        if (r0 > 0 && 16 * r0 >= rows) break;
        v8bf a[kPair][4];
        v4f p[kPair][C];
#pragma unroll
        for (int r = 0; r < kPair; ++r) {
            widen(k.a[r0 + r], a[r]);
#pragma unroll
            for (int c = 0; c < C; ++c) p[r][c] = v4f{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int r = 0; r < kPair; ++r)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    p[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[c][s], a[r][s], p[r][c], 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kPair; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if constexpr (kE8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[r0 + r][c][q] += scale_e8(p[r][c][q], k.sa[r0 + r], k.sb[c]);
                } else {
                    acc[r0 + r][c] += (k.sa[r0 + r] * k.sb[c]) * p[r][c];
                }
            }
    }
}

// acc += this block's scaled product; `rows` (uniform) of the 16 R rows count.
// The FP8 instruction, as in the dense form, whose sum this is to be: a row takes
// the same sum in either form, to about 16 bits of a K block's largest product.
// (multiply_exact here: 64 rows of 2112 x 7168 with adapters 17.6 -> 18.7 us,
// 1024 rows of 7168 x 2048 69 -> 85; the dense tiles would halve their rate.)
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

// ------------------------------------------------------------------- panels
//
// A workgroup of eight waves multiplies 16 R rows of A, shared, by 128 C rows
// of B, 16 C a wave.  A K block of all of it is one stage of a ring in LDS,
// filled by direct loads that take whole 128-byte lines, eight consecutive
// lanes a line: fragment-shaped loads straight to registers touch 16 lines
// for 16 bytes each and are bound by the cache's tag rate.  Each stage costs
// one barrier.  The stages ahead keep the weights of D - 1 K blocks in flight.
// In LDS 16-byte chunk c of row r sits at c ^ (r & 7), which the loading lanes
// arrange by the chunk they ask for, so that fragment reads do not conflict.
constexpr int kPanelWaves = 8;

template <int R, int C>
struct PanelStage {
    uint8_t b[kPanelWaves * C * 2048];  // wave w: C tiles of 16 rows
    uint8_t a[16 * R * 128];
    float sa[R > 4 ? 16 * R : 64];  // per row of A
    float sb[64];  // [c] of tile set c
};

// Bytes of LDS for a panel: the ring and the place where loads land that carry
// nothing (every wave issues the same number of loads per stage).
template <int R, int C, int D>
constexpr size_t panel_lds() {
    return D * sizeof(PanelStage<R, C>) + 1024;
}

// What the lanes of a wave load.  Offsets are bytes from the buffers' starts
// at K block 0, or kNoRow.
template <int C>
struct PanelLoads {
    v4u bufB, bufA, bufS;  // bufS: the scales this wave loads
    uint32_t offB[2 * C];  // lane l: row 8 j + l / 8 of the wave's 16 C rows
    uint32_t offA[4];      // lane l of wave w: rows of A, see panel_a_loads
    uint32_t offS;         // lane l of wave 0 (2): scale row l (64 + l) of A; of wave 1: column scales of tile set l
};

// Direct loads of a wave for the A rows of a panel's K block, or of a free
// panel's chunk; load i = wave * this + j takes rows 8 (i % 2R) .. + 7, and
// there may be more waves than loads.
constexpr int kChunk = 4;  // K blocks of a free panel's chunk
constexpr int panel_a_loads(int R, int W, int blocks) { return 2 * R * blocks > W ? 2 * R * blocks / W : 1; }

// The 16-byte chunk that lane l asks for, in bytes.
__device__ __forceinline__ uint32_t panel_chunk(int lane) { return ((lane & 7) ^ (lane >> 3)) * 16; }

// acc = the scaled product over KB K blocks; `rows` (uniform) rows of A count.
// kExact: through bf16 (multiply_exact).  The ring must be free on entry and
// is free again on return (the call ends with a barrier).
template <int R, int C, int D, bool kE8, bool kExact>
__device__ __forceinline__ void panel_product(uint8_t* smem, const PanelLoads<C>& p, int KB, int rows,
                                              int wave, int lane, v4f (&acc)[R][C]) {
    using Stage = PanelStage<R, C>;
    Stage* const ring = reinterpret_cast<Stage*>(smem);
    uint8_t* const unused = smem + D * sizeof(Stage);
    constexpr int kA = panel_a_loads(R, kPanelWaves, 1), kLoads = 2 * C + kA + 1;
    const int lr = lane & 15, lg = lane >> 4;
    auto issue = [&](int kb, Stage& s) __attribute__((always_inline)) {
        const bool real = kb < KB;  // stages past the last one load nothing
#pragma unroll
        for (int j = 0; j < 2 * C; ++j)
            load_lds_16(p.bufB, real ? p.offB[j] + kb * 128 : kNoRow, s.b + wave * C * 2048 + j * 1024);
#pragma unroll
        for (int j = 0; j < kA; ++j) {
            const int i = wave * kA + j;
            load_lds_16(p.bufA, real ? p.offA[j] + kb * 128 : kNoRow, i < 2 * R ? s.a + i * 1024 : unused);
        }
        load_lds_4(p.bufS, real ? p.offS + (kE8 ? kb & ~3 : kb * 4) : kNoRow,
                   wave == 0             ? (void*)s.sa
                   : wave == 1           ? (void*)s.sb
                   : R > 4 && wave == 2  ? (void*)(s.sa + 64)
                                         : (void*)unused);
    };
    clear(acc);
#pragma unroll
    for (int d = 0; d < D - 1; ++d) issue(d, ring[d]);
    const int lo = (lg ^ (lr & 7)) << 4, hi = lo ^ 64;
    int at = 0;
    for (int kb = 0; kb < KB; ++kb) {
        // stage kb has landed for this wave, and with the barrier for all; all
        // are also done with stage kb - 1, which the next loads refill
        wait_vmcnt_lgkm0<kLoads * (D - 2)>();
        lds_barrier();
        issue(kb + D - 1, ring[at == 0 ? D - 1 : at - 1]);
        const Stage& s = ring[at];
        Block<R, C, kE8> f;
        const uint8_t* const pb = s.b + wave * C * 2048 + lr * 128;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            f.b[c][0] = *reinterpret_cast<const v4u*>(pb + c * 2048 + lo);
            f.b[c][1] = *reinterpret_cast<const v4u*>(pb + c * 2048 + hi);
            if constexpr (kE8)  // one word holds four K blocks' exponents
                f.sb[c] = reinterpret_cast<const uint8_t*>(s.sb + c)[kb & 3];
            else
                f.sb[c] = s.sb[c];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            f.a[r][0] = *reinterpret_cast<const v4u*>(s.a + r * 2048 + lr * 128 + lo);
            f.a[r][1] = *reinterpret_cast<const v4u*>(s.a + r * 2048 + lr * 128 + hi);
            if constexpr (kE8)
                f.sa[r] = reinterpret_cast<const uint8_t*>(s.sa + 16 * r + lr)[kb & 3];
            else
                f.sa[r] = s.sa[16 * r + lr];
        }
        if constexpr (kExact)
            multiply_exact(f, rows, acc);
        else
            multiply(f, rows, acc);
        at = at == D - 1 ? 0 : at + 1;
    }
    wait_vmcnt_lgkm0<0>();  // the empty loads of the last stages have retired
    lds_barrier();
}

// For few rows of A the same panel without a barrier per K block: A and the
// scales come in chunks of four K blocks, double-buffered, one barrier per
// chunk; in between every wave runs on its own through its private ring of B.
// A wave waits for its loads in order, so waiting for the next chunk leaves at
// most the four K blocks of B behind it in flight: deeper rings gain nothing.
template <int R, int C, int D, int W>
struct FreePanel {
    static_assert(W >= 2, "wave 0 loads the row scales, wave 1 the column scales");
    uint8_t b[D][W * C * 2048];
    uint8_t a[2][kChunk][16 * R * 128];
    float sa[2][256];  // [row][kChunk]; E8M0: one word per row
    float sb[2][256];  // [c][kChunk]
    uint8_t unused[1024];
};

// `trips` chunks are walked (all waves of the workgroup alike), of which the
// first KB K blocks exist.
template <int R, int C, int D, int W, bool kE8>
__device__ __forceinline__ void free_panel_product(uint8_t* smem, const PanelLoads<C>& p, int KB, int trips,
                                                   int rows, int wave, int lane, v4f (&acc)[R][C]) {
    static_assert(R <= 2, "A chunks of more rows do not fit beside the ring");
    constexpr int kA = panel_a_loads(R, W, kChunk);
    static_assert(kA * W == 2 * R * kChunk, "every load of a chunk has a wave");
    FreePanel<R, C, D, W>& s = *reinterpret_cast<FreePanel<R, C, D, W>*>(smem);
    const int lr = lane & 15, lg = lane >> 4;
    auto issue_b = [&](int kb, int st) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2 * C; ++j)
            load_lds_16(p.bufB, kb < KB ? p.offB[j] + kb * 128 : kNoRow, s.b[st] + wave * C * 2048 + j * 1024);
    };
    // a wave's loads of an A chunk: K block i / 2R, rows 8 (i % 2R) .. + 7
    auto issue_chunk = [&](int kb0, int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kA; ++j) {
            const int i = wave * kA + j, kb = kb0 + i / (2 * R);
            load_lds_16(p.bufA, kb < KB ? p.offA[j] + kb * 128 : kNoRow, s.a[buf][0] + i * 1024);
        }
        void* const to = wave == 0 ? (void*)s.sa[buf] : wave == 1 ? (void*)s.sb[buf] : (void*)s.unused;
        const uint32_t off = kb0 < KB ? p.offS + kb0 * (kE8 ? 1 : 4) : kNoRow;
        if (kE8)
            load_lds_4(p.bufS, off, to);
        else
            load_lds_16(p.bufS, off, to);
    };
    clear(acc);
    issue_chunk(0, 0);
#pragma unroll
    for (int d = 0; d < D - 1; ++d) issue_b(d, d);
    wait_vmcnt_lgkm0<2 * C * (D - 1)>();
    lds_barrier();
    const int lo = (lg ^ (lr & 7)) << 4, hi = lo ^ 64;
    int at = 0, buf = 0;
    for (int kb0 = 0; kb0 < trips * kChunk; kb0 += kChunk) {
        issue_chunk(kb0 + kChunk, buf ^ 1);  // its last readers passed the barrier below
#pragma unroll
        for (int kk = 0; kk < kChunk; ++kk) {
            const int kb = kb0 + kk;
            if (kb < KB) {
                wait_vmcnt_lgkm0<2 * C * (D - 2)>();  // this wave's B of kb
                asm volatile("" ::: "memory");
                issue_b(kb + D - 1, at == 0 ? D - 1 : at - 1);
                Block<R, C, kE8> f;
                const uint8_t* const pb = s.b[at] + wave * C * 2048 + lr * 128;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    f.b[c][0] = *reinterpret_cast<const v4u*>(pb + c * 2048 + lo);
                    f.b[c][1] = *reinterpret_cast<const v4u*>(pb + c * 2048 + hi);
                    if constexpr (kE8)
                        f.sb[c] = reinterpret_cast<const uint8_t*>(s.sb[buf] + c)[kk];
                    else
                        f.sb[c] = s.sb[buf][c * kChunk + kk];
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const uint8_t* const pa = s.a[buf][kk] + (16 * r + lr) * 128;
                    f.a[r][0] = *reinterpret_cast<const v4u*>(pa + lo);
                    f.a[r][1] = *reinterpret_cast<const v4u*>(pa + hi);
                    if constexpr (kE8)
                        f.sa[r] = reinterpret_cast<const uint8_t*>(s.sa[buf] + 16 * r + lr)[kk];
                    else
                        f.sa[r] = s.sa[buf][(16 * r + lr) * kChunk + kk];
                }
                multiply_exact(f, rows, acc);
                at = at == D - 1 ? 0 : at + 1;
            }
        }
        wait_vmcnt_lgkm0<2 * C * kChunk>();  // the next chunk, loaded before these K blocks' B
        lds_barrier();
        buf ^= 1;
    }
    wait_vmcnt_lgkm0<0>();
    lds_barrier();
}

// Scales per row of `kb` K blocks: fp32 as they are, E8M0 bytes padded to four.
template <bool kE8>
__host__ __device__ __forceinline__ int scale_pitch(int kb) {
    return kE8 ? (kb + 3) & ~3 : kb;
}

}  // namespace dg
