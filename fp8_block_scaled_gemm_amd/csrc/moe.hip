// A whole gated expert layer for a few tokens.  include/dg_ops.h has the
// definition.
//
// Floor: the weights of the experts in use, 3 H I bytes each, read once;
// everything else is small.  Experts of 7168 x 2048: one token of 8 of them
// 69 us in two launches (352 MB, 5.1 TB/s); 64 tokens, 16 experts, 148 us in
// three (704 MB, 4.8 TB/s), where a large copy moves 5.04 TB/s.
//
// The routed pairs (token, choice) are kept in expert order ("routed rows"):
// row start_e + i is the i-th pair of expert e.  A unit is one expert's rows;
// units are numbered by expert, or, when there are fewer pairs than experts,
// by the first pair that names the expert.
#include "ops_launch.h"

#include <algorithm>
#include <type_traits>

#include "fewrow.h"
#include "quantize_common.h"
#include "wave_ops.h"

namespace dg {

struct MoeUnit {
    int e, start, count, pad;
};

// Up to 16 R rows of one unit.
struct MoeJob {
    int e;
    uint16_t start, count;
};

// LDS of the second product of a few pairs.
constexpr int kDownWaves = 8, kDownRing = 3;

struct MoeDownLds {
    int ring, codes, scales, cols, slices, row_w, jobs, row_t, total;
    __host__ __device__ MoeDownLds(int T, int P, int U, int I) {
        ring = 0;
        codes = kDownWaves * kDownRing * 2048;        // [P][I], chunk c of row r at c ^ (r & 7)
        scales = codes + P * I;                       // [P][I / 128]
        cols = scales + P * (I >> 7) * 4;             // [jobs][I / 128]
        slices = cols + (U + P / 16) * (I >> 7) * 4;  // [wave][T][16]
        slices = (slices + 15) & ~15;
        row_w = slices + kDownWaves * T * 64;
        jobs = row_w + ((P + 1) & ~1) * 4;
        row_t = jobs + (U + P / 16) * (int)sizeof(MoeJob);
        total = row_t + P * 2;
    }
};

// A few pairs: the hidden rows fit half a CU's LDS in the second product (so
// that two of its workgroups share a CU), which quantizes
// them for itself and adds up each token's experts (two launches), and the
// first product takes a part of a 128-column block a workgroup, as there are
// fewer blocks than CUs.  More pairs: 128 columns quantized by the first
// product, the second writes every pair's product, a third launch adds them up.
// (2 tokens, 8 experts of 7168 x 2048 as a few pairs: 124 us instead of 104.)
inline bool few_pairs(int64_t T, int64_t k, int64_t E, int64_t I) {
    const int64_t P = T * k, U = std::min(P, E);
    return T <= 16 && P * I <= 32768 && MoeDownLds((int)T, (int)P, (int)U, (int)I).total <= 80 * 1024;
}

// Workspace layout, in bytes from its start.
struct MoeLayout {
    int64_t units, order, place, codes, scales, hidden, out, total;
    MoeLayout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
        const int64_t P = T * k, U = std::min(P, E);
        auto up = [](int64_t v) { return (v + 255) & ~int64_t(255); };
        units = 0;
        order = units + up(U * sizeof(MoeUnit));
        place = order + up(P * 4);
        codes = place + up(P * 4);
        const bool few = few_pairs(T, k, E, I);
        scales = codes + (few ? 0 : up(P * I));
        hidden = scales + (few ? 0 : up(P * ((I / 128 + 3) & ~int64_t(3)) * 4));
        out = hidden + (few ? up(P * I * 4) : 0);
        total = out + (few ? 0 : up(P * H * 4));
    }
};

// Rows of one unit, found by the whole workgroup from the ids: the pairs of
// the unit's expert in order, into `list`.  count is 0 when the unit has no
// expert here, or (units numbered by pair) an earlier pair named it.  Each
// wave scans a share of the ids, copied to LDS first so that no step waits for
// memory.  `ids_lds` holds P ids and may be reused once this returns.
template <int W>
__device__ __forceinline__ MoeUnit find_unit(const int32_t* __restrict__ ids, int P, int E, int unit,
                                             bool by_pair, int* ids_lds, uint16_t* list) {
    __shared__ int found[W][3];  // pairs of the expert, pairs of lower experts, first pair
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int i = threadIdx.x; i < P; i += 64 * W) ids_lds[i] = ids[i];
    __syncthreads();
    MoeUnit u = {by_pair ? ids_lds[unit] : unit, 0, 0, 0};
    u.e = __builtin_amdgcn_readfirstlane(u.e);
    if (u.e < 0 || u.e >= E) return u;
    const int per = (P + 64 * W - 1) / (64 * W) * 64, q0 = wave * per, q1 = min(q0 + per, P);
    int count = 0, lower = 0, first = P;
    for (int base = q0; base < q1; base += 64) {
        const int id = base + lane < q1 ? ids_lds[base + lane] : -1;
        const uint64_t same = __ballot(id == u.e);
        if (count == 0 && same != 0) first = base + __builtin_ctzll(same);
        count += __popcll(same);
        lower += __popcll(__ballot(id >= 0 && id < u.e));
    }
    if (lane == 0) {
        found[wave][0] = count;
        found[wave][1] = lower;
        found[wave][2] = first;
    }
    __syncthreads();
    int before = 0, whole = 0;
    first = P;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w == wave) before = whole;
        whole += found[w][0];
        u.start += found[w][1];
        first = min(first, found[w][2]);
    }
    if (by_pair && first != unit) return u;
    u.count = __builtin_amdgcn_readfirstlane(whole);
    u.start = __builtin_amdgcn_readfirstlane(u.start);
    for (int base = q0; base < q1; base += 64) {
        const int id = base + lane < q1 ? ids_lds[base + lane] : -1;
        const uint64_t same = __ballot(id == u.e);
        if (id == u.e)
            list[before + __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0))] =
                (uint16_t)(base + lane);
        before += __popcll(same);
    }
    __syncthreads();
    return u;
}

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

// First product: silu(gate) * up, quantized per 128 hidden columns.  A
// workgroup takes one 128-column block of one unit, up to 16 R rows at a time;
// a wave multiplies its 16 gate and its 16 up rows of the weights by the same
// activations.
//
// The sums go through the bf16 matrix instruction (see multiply_exact): the
// FP8 one would move about one code in 600 of the quantized result.  Bound by
// the weights (470 MB of 16 experts for 64 tokens: 91 us, 5.2 TB/s).
//
// With four waves a workgroup takes 64 columns and leaves them in fp32, for
// the second product to quantize: for a few pairs there are too few 128
// column blocks to give every CU one, and a CU alone streams only 36 GB/s
// (8 pairs of 7168 x 2048: 51 us with 128 workgroups of 128 columns).
// A wave alone takes about 0.37 us per K block of 4 KB (reads, widening and
// products in sequence), so where even 64 columns leave CUs idle the workgroup
// takes fewer columns and KS groups of W waves split K.
template <int R, int D, int W, int KS>
constexpr size_t gate_lds() {
    if constexpr (R <= 2)
        return KS * sizeof(FreePanel<R, 2, D, W>);
    else
        return panel_lds<R, 2, D>();
}

template <int R, int D, int W, int KS, bool kE8>
__global__ __launch_bounds__(64 * W * KS) void moe_gate_up_kernel(
    const uint8_t* __restrict__ x, const void* __restrict__ sx_v, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ w13, const void* __restrict__ s13_v, MoeUnit* __restrict__ units,
    int32_t* __restrict__ order, int32_t* __restrict__ place, uint8_t* __restrict__ codes,
    void* __restrict__ scales, float* __restrict__ hidden, int P, int k, int E, int H, int I,
    bool by_pair) {
    using S = typename std::conditional<kE8, uint8_t, float>::type;
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr bool kFree = R <= 2;
    static_assert(W == kPanelWaves || kFree, "whole 128-column blocks, or a part of one in fp32");
    constexpr int kA = panel_a_loads(R, W, kFree ? kChunk : 1);
    uint16_t* const list = reinterpret_cast<uint16_t*>(smem + gate_lds<R, D, W, KS>());
    uint32_t* const tops = reinterpret_cast<uint32_t*>(smem);  // [16 R][W], once the ring is free
    static_assert(16 * R * W * 4 <= sizeof(PanelStage<R, 2>), "the magnitudes fit the ring");

    static_assert(KS == 1 || W < kPanelWaves, "K is split where there are few columns");
    const int lane = threadIdx.x & 63, at = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = at % W, share = at / W;  // this wave's columns, its share of K
    const int lr = lane & 15, lg = lane >> 4;
    const MoeUnit u = find_unit<W * KS>(ids, P, E, blockIdx.y, by_pair, reinterpret_cast<int*>(smem), list);
    if (blockIdx.x == 0 && threadIdx.x == 0) units[blockIdx.y] = u;
    if (u.count == 0) return;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < u.count; i += 64 * W * KS) {
            order[u.start + i] = list[i];
            place[list[i]] = u.start + i;
        }

    const int KB = H >> 7, SP = scale_pitch<kE8>(KB), NB = I >> 6;  // scale rows of w13: 2I / 128
    const int sub = lane >> 3, col = blockIdx.x * 16 * W + wave * 16;
    const uint32_t chunk = panel_chunk(lane), kSz = sizeof(S);
    // every offset fits 31 bits: 2 I H <= 2^29, T H <= 2^22
    PanelLoads<2> p;
    p.bufB = buffer_rsrc(w13 + (int64_t)u.e * 2 * I * H, (uint32_t)(2 * I) * (uint32_t)H);
    p.bufA = buffer_rsrc(x, (uint32_t)(P / k) * (uint32_t)H);
    p.bufS = wave != 1 ? buffer_rsrc(sx_v, (uint32_t)(P / k) * SP * kSz)
                       : buffer_rsrc(static_cast<const S*>(s13_v) + (int64_t)u.e * NB * SP, (uint32_t)NB * SP * kSz);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        p.offB[j] = (uint32_t)((j >> 1) * I + col + 8 * (j & 1) + sub) * (uint32_t)H + chunk;

    for (int m0 = 0; m0 < u.count; m0 += 16 * R) {
        const int rows = min(u.count - m0, 16 * R);
#pragma unroll
        for (int j = 0; j < kA; ++j) {
            const int arow = 8 * (kFree ? (wave * kA + j) % (2 * R) : wave * kA + j) + sub;
            p.offA[j] = arow < rows ? (uint32_t)(list[m0 + arow] / k) * (uint32_t)H + chunk : kNoRow;
        }
        const int srow = wave == 0 ? lane : R > 4 && wave == 2 ? 64 + lane : rows;  // whose scale this lane loads
        p.offS = srow < rows  ? (uint32_t)(list[m0 + srow] / k) * SP * kSz
                 : wave == 1 && lane < 2  ? (uint32_t)((lane * I + (int)blockIdx.x * 16 * W) >> 7) * SP * kSz
                                          : kNoRow;
        v4f acc[R][2];
        if constexpr (kFree) {
            using Panel = FreePanel<R, 2, D, W>;
            const int chunks = (KB + kChunk - 1) / kChunk, trips = (chunks + KS - 1) / KS, kb0 = share * trips * kChunk;
            PanelLoads<2> q = p;
            if (KS > 1) {
                q.offS += kb0 * kSz;
#pragma unroll
                for (int j = 0; j < kA; ++j) q.offA[j] += kb0 * 128;
#pragma unroll
                for (int j = 0; j < 4; ++j) q.offB[j] += kb0 * 128;
            }
            free_panel_product<R, 2, D, W, kE8>(
                smem + share * sizeof(Panel), q, min(max(KB - kb0, 0), trips * kChunk), trips, rows, wave, lane, acc);
            if constexpr (KS > 1) {
                // the shares' sums meet in LDS, in order; the ring is free
                v4f* const part = reinterpret_cast<v4f*>(smem);
                static_assert(KS * W * R * 2 * 64 * 16 <= gate_lds<R, D, W, KS>(), "the sums fit the ring");
                if (share > 0) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int c = 0; c < 2; ++c) part[((at * R + r) * 2 + c) * 64 + lane] = acc[r][c];
                }
                __syncthreads();
                if (share == 0) {
#pragma unroll
                    for (int s = 1; s < KS; ++s)
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                acc[r][c] += part[(((s * W + wave) * R + r) * 2 + c) * 64 + lane];
                }
                __syncthreads();
                if (share > 0) continue;
            }
        } else
            panel_product<R, 2, D, kE8, true>(smem, p, KB, rows, wave, lane, acc);

        v4f h[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float g = acc[r][0][q];
                h[r][q] = g / (1.0f + expf(-g)) * acc[r][1][q];
            }
        if constexpr (W != kPanelWaves) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (16 * r + lr < rows)
                    *reinterpret_cast<v4f*>(hidden + (int64_t)(u.start + m0 + 16 * r + lr) * I + col + 4 * lg) =
                        h[r];
            continue;
        }
        // the block's largest magnitude per row across the waves, compared as
        // bits so that a NaN wins
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t top = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) top = max(top, __float_as_uint(h[r][q]) & 0x7fffffffu);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
            if (lg == 0) tops[(16 * r + lr) * W + wave] = top;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = 16 * r + lr;
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < kPanelWaves; ++w) top = max(top, tops[row * W + w]);
            if (row >= rows) continue;
            uint32_t packed;
            const auto scale = quantize_hidden<kE8>(top, h[r], packed);
            const int64_t out = u.start + m0 + row;
            *reinterpret_cast<uint32_t*>(codes + out * I + col + 4 * lg) = packed;
            if (wave == 0 && lg == 0)
                static_cast<S*>(scales)[out * scale_pitch<kE8>(I >> 7) + blockIdx.x] = (S)scale;
        }
        __syncthreads();  // tops have been read
    }
}

// Second product of a batch, unweighted: out[row] = h w2^T in fp32, one 128
// column block of one unit per workgroup.  Bound by the weights (235 MB for 64
// tokens, 16 experts: 50.8 us, 4.6 TB/s).  With the tokens' weighted sum in
// the same launch, which has to gather a column block's experts in one
// workgroup, it took 134 us.
template <int R, int D, bool kE8>
__global__ __launch_bounds__(64 * kPanelWaves) void moe_down_rows_kernel(
    const uint8_t* __restrict__ codes, const void* __restrict__ sh_v, const uint8_t* __restrict__ w2,
    const void* __restrict__ s2_v, const MoeUnit* __restrict__ units, float* __restrict__ out, int P,
    int H, int I) {
    using S = typename std::conditional<kE8, uint8_t, float>::type;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int e = __builtin_amdgcn_readfirstlane(units[blockIdx.y].e);
    const int start = __builtin_amdgcn_readfirstlane(units[blockIdx.y].start);
    const int count = __builtin_amdgcn_readfirstlane(units[blockIdx.y].count);
    const int KB = I >> 7, SP = scale_pitch<kE8>(KB), NB = H >> 7;
    const int sub = lane >> 3, col = blockIdx.x * 128 + wave * 16;
    const uint32_t chunk = panel_chunk(lane), kSz = sizeof(S);
    for (int m0 = 0; m0 < count; m0 += 16 * R) {
        const int rows = min(count - m0, 16 * R), row0 = start + m0;
        PanelLoads<1> p;
        // offsets fit 31 bits: H I <= 2^28, 16 R rows of I
        p.bufB = buffer_rsrc(w2 + (int64_t)e * H * I, (uint32_t)H * (uint32_t)I);
        p.bufA = buffer_rsrc(codes + (int64_t)row0 * I, (uint32_t)rows * (uint32_t)I);
        p.bufS = wave != 1
                     ? buffer_rsrc(static_cast<const S*>(sh_v) + (int64_t)row0 * SP, (uint32_t)rows * SP * kSz)
                     : buffer_rsrc(static_cast<const S*>(s2_v) + (int64_t)e * NB * SP, (uint32_t)NB * SP * kSz);
#pragma unroll
        for (int j = 0; j < 2; ++j) p.offB[j] = (uint32_t)(col + 8 * j + sub) * (uint32_t)I + chunk;
#pragma unroll
        for (int j = 0; j < panel_a_loads(R, kPanelWaves, 1); ++j) {
            const int arow = 8 * (wave * panel_a_loads(R, kPanelWaves, 1) + j) + sub;
            p.offA[j] = arow < rows ? (uint32_t)arow * (uint32_t)I + chunk : kNoRow;
        }
        const int srow = wave == 0 ? lane : R > 4 && wave == 2 ? 64 + lane : rows;  // whose scale this lane loads
        p.offS = srow < rows                ? (uint32_t)srow * SP * kSz
                 : wave == 1 && lane == 0 ? (uint32_t)blockIdx.x * SP * kSz
                                          : kNoRow;
        v4f acc[R][1];
        panel_product<R, 1, D, kE8, true>(smem, p, KB, rows, wave, lane, acc);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (16 * r + lr < rows)
                *reinterpret_cast<v4f*>(out + (int64_t)(row0 + 16 * r + lr) * H + col + 4 * lg) = acc[r][0];
    }
}

// y_t = bf16(sum over j of weight * out[place of (t, j)]), four columns a
// thread; one rounding, after the whole sum.  Bound by latency: 15 MB from L2
// and beyond for 64 tokens, 5.6 us.
__global__ __launch_bounds__(256) void moe_combine_kernel(const float* __restrict__ out,
                                                          const int32_t* __restrict__ ids,
                                                          const int32_t* __restrict__ place,
                                                          const float* __restrict__ weights,
                                                          uint16_t* __restrict__ y, int k, int E, int H) {
    const int64_t t = blockIdx.y;
    const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= H) return;
    v4f sum = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < k; ++j) {
        const int id = ids[t * k + j];
        if (id < 0 || id >= E) continue;
        sum += weights[t * k + j] * *reinterpret_cast<const v4f*>(out + (int64_t)place[t * k + j] * H + c);
    }
    const v2f lo = {sum[0], sum[1]}, hi = {sum[2], sum[3]};
    v2u packed;
    packed[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, v2bf));
    packed[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, v2bf));
    *reinterpret_cast<v2u*>(y + t * H + c) = packed;
}

// Second product of a few pairs with the weighted sum: a workgroup owns 16
// columns of y for every token.  It quantizes the hidden rows into LDS for
// itself (at most 32 K values, from L2, behind the first weights), then its
// waves split the list of (up to 16 rows of an expert, K block) steps evenly,
// each streaming its share of the weights through a ring of its own in LDS,
// with no barrier.  A wave adds its weighted products to a slice of its own
// ([token][16] fp32); the slices are summed in wave order at the end.
// One token, 8 experts of 7168 x 2048: 26.5 us for 117 MB (4.4 TB/s), of which
// about 5 us pass before the first product (ids, hidden rows, first weights,
// one load's latency after the other).
template <bool kE8>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_kernel(
    const float* __restrict__ hidden, const float* __restrict__ weights, const uint8_t* __restrict__ w2,
    const void* __restrict__ s2_v, const MoeUnit* __restrict__ units, const int32_t* __restrict__ order,
    uint16_t* __restrict__ y, int T, int U, int k, int H, int I) {
    constexpr int W = kDownWaves, D = kDownRing;
    using S = typename std::conditional<kE8, uint8_t, float>::type;
    using V = typename std::conditional<kE8, int, float>::type;
    const S* s2 = static_cast<const S*>(s2_v);
    extern __shared__ __align__(1024) uint8_t smem[];
    const int P = T * k;
    const MoeDownLds at(T, P, U, I);
    uint8_t* const codes = smem + at.codes;
    V* const scales = reinterpret_cast<V*>(smem + at.scales);
    V* const cols = reinterpret_cast<V*>(smem + at.cols);
    float* const slices = reinterpret_cast<float*>(smem + at.slices);
    float* const row_w = reinterpret_cast<float*>(smem + at.row_w);
    MoeJob* const jobs = reinterpret_cast<MoeJob*>(smem + at.jobs);
    uint16_t* const row_t = reinterpret_cast<uint16_t*>(smem + at.row_t);
    __shared__ int totals[2];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    // What does not depend on the units is asked for first: the hidden values,
    // 8 a thread at a time, and the rows' pairs (of all P places; those past
    // the routed rows hold nothing meaningful and are not used).  A wave waits
    // for its loads in order, so all of this is consumed before the weights'
    // ring starts: the other way round the weights' first stages, from HBM,
    // stand in front of it and then the ring runs dry (25.7 instead of 25.1 us).
    constexpr int kBatch = 4;
    const int per_row = I >> 3, places = P * per_row;
    v4f v[kBatch][2];
    auto fetch = [&](int base) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            const float* const from = hidden + (int64_t)min(base + n * 64 * W + (int)threadIdx.x, places - 1) * 8;
            v[n][0] = *reinterpret_cast<const v4f*>(from);
            v[n][1] = *reinterpret_cast<const v4f*>(from + 4);
        }
    };
    int pair = 0;  // of row threadIdx.x: P <= 16 * 16
    if ((int)threadIdx.x < P) pair = order[threadIdx.x];
    fetch(0);
    if (wave == 0) {
        int n = 0, rows = 0;
        for (int base = 0; base < U; base += 64) {
            MoeUnit u = {0, 0, 0, 0};
            if (base + lane < U) u = units[base + lane];
            const int c = (u.count + 15) / 16;
            int sum_c = c, sum_r = u.count;  // inclusive sums over the lanes
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int oc = __shfl_up(sum_c, d, 64), orow = __shfl_up(sum_r, d, 64);
                if (lane >= d) {
                    sum_c += oc;
                    sum_r += orow;
                }
            }
            for (int i = 0; i < c; ++i)
                jobs[n + sum_c - c + i] = MoeJob{u.e, (uint16_t)(u.start + 16 * i), (uint16_t)min(16, u.count - 16 * i)};
            n += __shfl(sum_c, 63, 64);
            rows += __shfl(sum_r, 63, 64);
        }
        if (lane == 0) {
            totals[0] = n;
            totals[1] = rows;
        }
    }
    for (int i = threadIdx.x; i < W * T * 16; i += 64 * W) slices[i] = 0.0f;
    __syncthreads();
    const int n_jobs = __builtin_amdgcn_readfirstlane(totals[0]);
    const int n_rows = __builtin_amdgcn_readfirstlane(totals[1]);
    const int KB = I >> 7, SP = scale_pitch<kE8>(KB), n0 = blockIdx.x * 16, NB = H >> 7;
    const int items = n_rows * per_row;
    // 16 lanes quantize one 128-column block of one row, 8 columns each
    // (a thread's next place is 64 W eights further on: one division in all)
    int row = (int)threadIdx.x / per_row, c = (int)threadIdx.x - row * per_row;
    for (int base = 0; base < items; base += kBatch * 64 * W) {
        if (base > 0) fetch(base);
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            if (row >= n_rows) break;  // uniform over each 16 lanes
            uint32_t top = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[n][q >> 2][q & 3]) & 0x7fffffffu);
            top = row_max(top);
            uint32_t w[2];
            const V s = quantize_hidden<kE8>(top, v[n][0], w[0]);
            quantize_hidden<kE8>(top, v[n][1], w[1]);
            const int in = (c & 15) * 8;  // byte in the 128-byte block
            uint8_t* const to = codes + row * I + (c >> 4) * 128 + ((((in >> 4) ^ row) & 7) << 4) + (in & 15);
            *reinterpret_cast<v2u*>(to) = v2u{w[0], w[1]};
            if ((c & 15) == 0) scales[row * KB + (c >> 4)] = s;
            for (c += 64 * W; c >= per_row; c -= per_row) ++row;
        }
    }

    const int first = wave * n_jobs * KB / W, last = (wave + 1) * n_jobs * KB / W;

    // the loader runs D - 1 steps ahead of the multiplier, each with its own
    // place (job, K block) in the list; past the wave's share it loads nothing
    uint8_t* const ring = smem + at.ring + wave * D * 2048;
    const uint32_t off0 = (uint32_t)(n0 + (lane >> 3)) * (uint32_t)I + panel_chunk(lane);
    int lj = KB > 0 && n_jobs > 0 ? first / KB : 0, lk = first - lj * KB, ls = first;
    v4u buf = buffer_rsrc(w2, 0);
    if (ls < last)
        buf = buffer_rsrc(w2 + (int64_t)__builtin_amdgcn_readfirstlane(jobs[lj].e) * H * I, (uint32_t)H * (uint32_t)I);
    auto issue = [&](int slot) __attribute__((always_inline)) {
        const bool real = ls < last;
        load_lds_16(buf, real ? off0 + lk * 128 : kNoRow, ring + slot * 2048);
        load_lds_16(buf, real ? off0 + 8 * I + lk * 128 : kNoRow, ring + slot * 2048 + 1024);
        ++ls;
        if (++lk == KB) {
            lk = 0;
            ++lj;
            if (ls < last)
                buf = buffer_rsrc(w2 + (int64_t)__builtin_amdgcn_readfirstlane(jobs[lj].e) * H * I,
                                  (uint32_t)H * (uint32_t)I);
        }
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) issue(d);
    // needed with the first weights, so behind them
    if ((int)threadIdx.x < n_rows) {
        row_w[threadIdx.x] = weights[pair];
        row_t[threadIdx.x] = (uint16_t)(pair / k);
    }
    for (int i = threadIdx.x; i < n_jobs * KB; i += 64 * W)
        cols[i] = s2[((int64_t)jobs[i / KB].e * NB + (n0 >> 7)) * SP + i % KB];
    wait_vmcnt_lgkm0<63>();  // LDS is written; the ring stays in flight
    lds_barrier();

    float* const mine = slices + wave * T * 16;
    const int lo = (lg ^ (lr & 7)) << 4, hi = lo ^ 64;
    int j = first < last ? first / KB : 0, kb = first - j * KB, slot = 0;
    v4f acc[1][1];
    clear(acc);
    for (int s = first; s < last; ++s) {
        wait_vmcnt_lgkm0<2 * (D - 2)>();
        asm volatile("" ::: "memory");
        issue(slot == 0 ? D - 1 : slot - 1);
        const int count = __builtin_amdgcn_readfirstlane(jobs[j].count);
        const int start = __builtin_amdgcn_readfirstlane(jobs[j].start);
        const int row = start + min(lr, count - 1);
        const uint8_t* const pb = ring + slot * 2048 + lr * 128;
        const uint8_t* const pa = codes + row * I + kb * 128;
        Block<1, 1, kE8> f;
        f.b[0][0] = *reinterpret_cast<const v4u*>(pb + lo);
        f.b[0][1] = *reinterpret_cast<const v4u*>(pb + hi);
        f.a[0][0] = *reinterpret_cast<const v4u*>(pa + ((lg ^ (row & 7)) << 4));
        f.a[0][1] = *reinterpret_cast<const v4u*>(pa + (((lg + 4) ^ (row & 7)) << 4));
        f.sa[0] = scales[row * KB + kb];
        f.sb[0] = cols[j * KB + kb];
        multiply_exact(f, 16, acc);
        slot = slot == D - 1 ? 0 : slot + 1;
        if (++kb == KB || s + 1 == last) {
            const v4f part = row_w[row] * acc[0][0];
            const int t = row_t[row];
            float* const to = mine + t * 16 + 4 * lg;
            // rows of one token (an expert listed more than once) are adjacent;
            // they are added one after the other, so that the order is fixed
            const bool again = lr > 0 && lr < count && row_t[row - 1] == t;
            if (__ballot(again) == 0) {
                if (lr < count) *reinterpret_cast<v4f*>(to) += part;
                wave_sync();
            } else {
                for (int r = 0; r < count; ++r) {
                    if (lr == r) *reinterpret_cast<v4f*>(to) += part;
                    wave_sync();
                }
            }
            clear(acc);
            kb = 0;
            ++j;
        }
    }
    wait_vmcnt_lgkm0<0>();  // the empty loads of the last steps have retired
    __syncthreads();
    for (int i = threadIdx.x; i < T * 8; i += 64 * W) {
        const int t = i >> 3, c = (i & 7) * 2;
        v2f s = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) s += *reinterpret_cast<const v2f*>(slices + (w * T + t) * 16 + c);
        *reinterpret_cast<uint32_t*>(y + (int64_t)t * H + n0 + c) =
            __builtin_bit_cast(uint32_t, __builtin_convertvector(s, v2bf));
    }
}

int64_t moe_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
    return MoeLayout(T, k, E, H, I).total;
}

// Whether a launch's dynamic LDS fits a CU's 160 KB beside a kernel's own few
// hundred bytes (rounded up to 1 KB): a launch past it would abort the queue.
static bool lds_fits(size_t bytes) { return bytes + 1024 <= 160 * 1024; }

template <bool kE8>
static dg_status moe_few(const MoeArgs& a, hipStream_t stream) {
    const MoeLayout at(a.T, a.k, a.E, a.H, a.I);
    uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
    MoeUnit* const units = reinterpret_cast<MoeUnit*>(ws + at.units);
    int32_t* const order = reinterpret_cast<int32_t*>(ws + at.order);
    float* const hidden = reinterpret_cast<float*>(ws + at.hidden);
    const int P = a.T * a.k, U = std::min(P, a.E);
    auto first = [&](auto waves, auto shares, auto depth) {
        constexpr int W = decltype(waves)::value, KS = decltype(shares)::value, D = decltype(depth)::value;
        static_assert(gate_lds<1, D, W, KS>() + 512 + 1024 <= 160 * 1024, "P <= 16 * 16");
        hipLaunchKernelGGL((moe_gate_up_kernel<1, D, W, KS, kE8>), dim3(a.I / (16 * W), U), dim3(64 * W * KS),
                           (gate_lds<1, D, W, KS>()) + P * 2, stream, a.x, a.sx, a.ids, a.w13, a.s13, units, order,
                           reinterpret_cast<int32_t*>(ws + at.place), nullptr, nullptr, hidden, P, a.k, a.E, a.H,
                           a.I, P <= a.E);
    };
    const size_t down_lds = MoeDownLds(a.T, P, U, a.I).total;
    if (!lds_fits(down_lds)) return DG_ERR_UNSUPPORTED;
    using std::integral_constant;
    // 2 pairs of 4096 x 1792, 112 workgroups of 32 columns: 11.5 us with K in
    // two shares, 17.8 with K whole
    if (U * (a.I / 64) >= 192)
        first(integral_constant<int, 4>{}, integral_constant<int, 1>{}, integral_constant<int, 4>{});
    else
        first(integral_constant<int, 2>{}, integral_constant<int, 2>{}, integral_constant<int, 5>{});
    if (launched() != DG_OK) return DG_ERR_HIP;
    hipLaunchKernelGGL((moe_down_kernel<kE8>), dim3(a.H / 16), dim3(64 * kDownWaves),
                       down_lds, stream, hidden, a.weights, a.w2, a.s2, units, order,
                       a.y, a.T, U, a.k, a.H, a.I);
    return launched();
}

template <int R, bool kE8>
static dg_status moe_many(const MoeArgs& a, hipStream_t stream) {
    const MoeLayout at(a.T, a.k, a.E, a.H, a.I);
    uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
    MoeUnit* const units = reinterpret_cast<MoeUnit*>(ws + at.units);
    int32_t* const place = reinterpret_cast<int32_t*>(ws + at.place);
    float* const out = reinterpret_cast<float*>(ws + at.out);
    const int P = a.T * a.k, U = std::min(P, a.E);
    constexpr int D = R == 1 ? 4 : 3, D2 = R == 8 ? 2 : 3;
    const size_t gate = gate_lds<R, D, kPanelWaves, 1>() + P * 2;
    if (!lds_fits(gate) || !lds_fits(panel_lds<R, 1, D2>())) return DG_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((moe_gate_up_kernel<R, D, kPanelWaves, 1, kE8>), dim3(a.I / 128, U), dim3(64 * kPanelWaves),
                       gate, stream, a.x, a.sx, a.ids, a.w13, a.s13, units,
                       reinterpret_cast<int32_t*>(ws + at.order), place, ws + at.codes, ws + at.scales, nullptr,
                       P, a.k, a.E, a.H, a.I, P <= a.E);
    if (launched() != DG_OK) return DG_ERR_HIP;
    hipLaunchKernelGGL((moe_down_rows_kernel<R, D2, kE8>), dim3(a.H / 128, U), dim3(64 * kPanelWaves),
                       (panel_lds<R, 1, D2>()), stream, ws + at.codes, ws + at.scales, a.w2, a.s2, units, out, P,
                       a.H, a.I);
    if (launched() != DG_OK) return DG_ERR_HIP;
    hipLaunchKernelGGL(moe_combine_kernel, dim3((a.H + 1023) / 1024, a.T), dim3(256), 0, stream, out, a.ids, place,
                       a.weights, a.y, a.k, a.E, a.H);
    return launched();
}

template <bool kE8>
static dg_status moe_scales(const MoeArgs& a, hipStream_t stream) {
    if (few_pairs(a.T, a.k, a.E, a.I)) return moe_few<kE8>(a, stream);
    if (a.T <= 16) return moe_many<1, kE8>(a, stream);
    if (a.T <= 32) return moe_many<2, kE8>(a, stream);
    // 128 rows at a time where an expert would have more than 64 if every pair
    // were routed here (256 tokens, 8 of 16 experts: 299 instead of 373 us;
    // with 16 rows an expert 140 instead of 137)
    if (a.T <= 64 || a.T * a.k <= 64 * a.E) return moe_many<4, kE8>(a, stream);
    return moe_many<8, kE8>(a, stream);
}

dg_status launch_moe(const MoeArgs& a, bool e8m0, hipStream_t stream) {
    return e8m0 ? moe_scales<true>(a, stream) : moe_scales<false>(a, stream);
}

}  // namespace dg
