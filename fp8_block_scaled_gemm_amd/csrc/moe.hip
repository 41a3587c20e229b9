// A whole gated expert layer for a few tokens.  include/dg_ops.h has the
// definition.
//
// Floor: the weights of the experts in use, 3 H I bytes each, read once;
// everything else is small.
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

namespace dg {

struct MoeUnit {
    int e, start, count, pad;
};

// Up to 16 R rows of one unit.
struct MoeJob {
    int e;
    uint16_t start, count;
};

// Up to this many tokens the second product adds up each token's experts
// itself; larger batches write every pair's product and add them up after.
constexpr int kFusedTokens = 16;

// Workspace layout, in bytes from its start.
struct MoeLayout {
    int64_t units, order, place, codes, scales, out, total;
    MoeLayout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
        const int64_t P = T * k, U = std::min(P, E);
        auto up = [](int64_t v) { return (v + 255) & ~int64_t(255); };
        units = 0;
        order = units + up(U * sizeof(MoeUnit));
        place = order + up(P * 4);
        codes = place + up(P * 4);
        scales = codes + up(P * I);
        out = scales + up(P * ((I / 128 + 3) & ~int64_t(3)) * 4);
        total = out + (T > kFusedTokens ? up(P * H * 4) : 0);
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

// First product: silu(gate) * up, quantized per 128 hidden columns.  A
// workgroup takes one 128-column block of one unit, up to 16 R rows at a time;
// a wave multiplies its 16 gate and its 16 up rows of the weights by the same
// activations.
//
// The sums go through the bf16 matrix instruction (see multiply_exact): the
// FP8 one would move about one code in 600 of the quantized result.
template <int R, int D, bool kE8>
__global__ __launch_bounds__(64 * kPanelWaves) void moe_gate_up_kernel(
    const uint8_t* __restrict__ x, const void* __restrict__ sx_v, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ w13, const void* __restrict__ s13_v, MoeUnit* __restrict__ units,
    int32_t* __restrict__ order, int32_t* __restrict__ place, uint8_t* __restrict__ codes,
    void* __restrict__ scales, int P, int k, int E, int H, int I, bool by_pair) {
    using S = typename std::conditional<kE8, uint8_t, float>::type;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint16_t* const list = reinterpret_cast<uint16_t*>(smem + panel_lds<R, 2, D>());
    __shared__ uint32_t tops[16 * R][kPanelWaves];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const MoeUnit u = find_unit<kPanelWaves>(ids, P, E, blockIdx.y, by_pair, reinterpret_cast<int*>(smem), list);
    if (blockIdx.x == 0 && threadIdx.x == 0) units[blockIdx.y] = u;
    if (u.count == 0) return;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < u.count; i += 64 * kPanelWaves) {
            order[u.start + i] = list[i];
            place[list[i]] = u.start + i;
        }

    const int KB = H >> 7, SP = scale_pitch<kE8>(KB), NB = I >> 6;  // scale rows of w13: 2I / 128
    const int sub = lane >> 3, col = blockIdx.x * 128 + wave * 16;
    const uint32_t chunk = panel_chunk(lane), kSz = sizeof(S);
    // every offset fits 31 bits: 2 I H <= 2^29, T H <= 2^22
    PanelLoads<2> p;
    p.bufB = buffer_rsrc(w13 + (int64_t)u.e * 2 * I * H, (uint32_t)(2 * I) * (uint32_t)H);
    p.bufA = buffer_rsrc(x, (uint32_t)(P / k) * (uint32_t)H);
    p.bufS = wave == 0 ? buffer_rsrc(sx_v, (uint32_t)(P / k) * SP * kSz)
                       : buffer_rsrc(static_cast<const S*>(s13_v) + (int64_t)u.e * NB * SP, (uint32_t)NB * SP * kSz);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        p.offB[j] = (uint32_t)((j >> 1) * I + col + 8 * (j & 1) + sub) * (uint32_t)H + chunk;

    for (int m0 = 0; m0 < u.count; m0 += 16 * R) {
        const int rows = min(u.count - m0, 16 * R), arow = 8 * wave + sub;
        p.offA = arow < rows ? (uint32_t)(list[m0 + arow] / k) * (uint32_t)H + chunk : kNoRow;
        p.offS = wave == 0 && lane < rows ? (uint32_t)(list[m0 + lane] / k) * SP * kSz
                 : wave == 1 && lane < 2  ? (uint32_t)((lane * I + blockIdx.x * 128) >> 7) * SP * kSz
                                          : kNoRow;
        v4f acc[R][2];
        panel_product<R, 2, D, kE8, true>(smem, p, KB, rows, wave, lane, acc);

        // silu(gate) * up, then the block's largest magnitude per row across
        // the waves, compared as bits so that a NaN wins
        float h[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t top = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float g = acc[r][0][q];
                h[r][q] = g / (1.0f + expf(-g)) * acc[r][1][q];
                top = max(top, __float_as_uint(h[r][q]) & 0x7fffffffu);
            }
            top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
            if (lg == 0) tops[16 * r + lr][wave] = top;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = 16 * r + lr;
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < kPanelWaves; ++w) top = max(top, tops[row][w]);
            if (row >= rows) continue;
            const float a = __uint_as_float(top);
            const bool finite = top < 0x7f800000u;
            const float scale = a / 448.0f;
            const int ex = kE8 ? e8m0_exponent(a) : 0;
            const float y = kE8 ? exp2_neg(ex) : 1.0f / scale;
            const bool fast = scale >= 1.17549435e-38f && y <= 3.40282347e38f;
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] = kE8 ? h[r][q] * y : fast ? quotient_rn(h[r][q], scale, y) : h[r][q] / scale;
            const int64_t out = u.start + m0 + row;
            *reinterpret_cast<uint32_t*>(codes + out * I + col + 4 * lg) =
                (kE8 || top != 0) ? e4m3x4_hw(v[0], v[1], v[2], v[3]) : 0u;
            if (wave == 0 && lg == 0) {
                const int64_t to = out * scale_pitch<kE8>(I >> 7) + blockIdx.x;
                if (kE8)
                    static_cast<uint8_t*>(scales)[to] = finite ? (uint8_t)(ex + 127) : (uint8_t)255;
                else
                    static_cast<float*>(scales)[to] = finite ? scale : __builtin_nanf("");
            }
        }
        __syncthreads();  // tops have been read
    }
}

// Second product of a batch, unweighted: out[row] = h w2^T in fp32, one 128
// column block of one unit per workgroup.
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
        const int rows = min(count - m0, 16 * R), arow = 8 * wave + sub, row0 = start + m0;
        PanelLoads<1> p;
        // offsets fit 31 bits: H I <= 2^28, 16 R rows of I
        p.bufB = buffer_rsrc(w2 + (int64_t)e * H * I, (uint32_t)H * (uint32_t)I);
        p.bufA = buffer_rsrc(codes + (int64_t)row0 * I, (uint32_t)rows * (uint32_t)I);
        p.bufS = wave == 0
                     ? buffer_rsrc(static_cast<const S*>(sh_v) + (int64_t)row0 * SP, (uint32_t)rows * SP * kSz)
                     : buffer_rsrc(static_cast<const S*>(s2_v) + (int64_t)e * NB * SP, (uint32_t)NB * SP * kSz);
#pragma unroll
        for (int j = 0; j < 2; ++j) p.offB[j] = (uint32_t)(col + 8 * j + sub) * (uint32_t)I + chunk;
        p.offA = arow < rows ? (uint32_t)arow * (uint32_t)I + chunk : kNoRow;
        p.offS = wave == 0 && lane < rows ? (uint32_t)lane * SP * kSz
                 : wave == 1 && lane == 0 ? (uint32_t)blockIdx.x * SP * kSz
                                          : kNoRow;
        v4f acc[R][1];
        panel_product<R, 1, D, kE8, false>(smem, p, KB, rows, wave, lane, acc);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (16 * r + lr < rows)
                *reinterpret_cast<v4f*>(out + (int64_t)(row0 + 16 * r + lr) * H + col + 4 * lg) = acc[r][0];
    }
}

// y_t = bf16(sum over j of weight * out[place of (t, j)]), four columns a thread.
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

// Second product and the weighted sum: a workgroup owns 16 columns of y for
// every token.  Its waves split the list of (16 R rows of an expert, K block)
// steps evenly and add their weighted products to an LDS slice of their own
// ([token][16] fp32); the slices are summed in wave order at the end.
template <int R, bool kE8, int W>
__global__ __launch_bounds__(64 * W) void moe_down_kernel(
    const uint8_t* __restrict__ codes, const void* __restrict__ sh_v, const float* __restrict__ weights,
    const uint8_t* __restrict__ w2, const void* __restrict__ s2_v, const MoeUnit* __restrict__ units,
    const int32_t* __restrict__ order, uint16_t* __restrict__ y, int T, int U, int k, int H, int I) {
    using S = typename std::conditional<kE8, uint8_t, float>::type;
    const S* sh = static_cast<const S*>(sh_v);
    const S* s2 = static_cast<const S*>(s2_v);
    extern __shared__ __align__(16) uint8_t smem[];
    const int P = T * k;
    float* const slices = reinterpret_cast<float*>(smem);                      // [W][T][16]
    float* const row_w = slices + W * T * 16;                                  // [P]
    MoeJob* const jobs = reinterpret_cast<MoeJob*>(row_w + ((P + 3) & ~3));  // [U + P / (16 R)]
    uint16_t* const row_t = reinterpret_cast<uint16_t*>(jobs + U + P / (16 * R));  // [P]
    __shared__ int totals[2];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    for (int i = threadIdx.x; i < W * T * 16; i += 64 * W) slices[i] = 0.0f;
    if (wave == 0) {
        int n = 0, rows = 0;
        for (int base = 0; base < U; base += 64) {
            MoeUnit u = {0, 0, 0, 0};
            if (base + lane < U) u = units[base + lane];
            const int c = (u.count + 16 * R - 1) / (16 * R);
            int at = c, sum = u.count;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(at, d, 64), s = __shfl_up(sum, d, 64);
                if (lane >= d) {
                    at += o;
                    sum += s;
                }
            }
            for (int i = 0; i < c; ++i)
                jobs[n + at - c + i] = MoeJob{u.e, (uint16_t)(u.start + 16 * R * i),
                                              (uint16_t)min(16 * R, u.count - 16 * R * i)};
            n += __shfl(at, 63, 64);
            rows += __shfl(sum, 63, 64);
        }
        if (lane == 0) {
            totals[0] = n;
            totals[1] = rows;
        }
    }
    __syncthreads();
    const int n_jobs = __builtin_amdgcn_readfirstlane(totals[0]);
    const int n_rows = __builtin_amdgcn_readfirstlane(totals[1]);
    for (int i = threadIdx.x; i < n_rows; i += 64 * W) {
        const int q = order[i];
        row_w[i] = weights[q];
        row_t[i] = (uint16_t)(q / k);
    }
    __syncthreads();

    const int KB = I >> 7, SP = scale_pitch<kE8>(KB), n0 = blockIdx.x * 16, NB = H >> 7;
    const int first = (int)((int64_t)wave * n_jobs * KB / W);
    const int last = (int)((int64_t)(wave + 1) * n_jobs * KB / W);
    float* const mine = slices + wave * T * 16;
    if (first < last) {
        constexpr int D = R == 1 ? 4 : 2;
        Block<R, 1, kE8> ring[D];
        // the loader runs D steps ahead of the multiplier, each with its own
        // place (job, K block) in the list
        int lj = first / KB, lk = first % KB;
        const auto hbuf = buffer_of(codes, (int64_t)P * I);
        const uint8_t* b;
        uint32_t a[R];
        const S *sb, *sa[R];
        auto aim = [&](int j) __attribute__((always_inline)) {
            const int e = __builtin_amdgcn_readfirstlane(jobs[j].e);
            const int start = __builtin_amdgcn_readfirstlane(jobs[j].start);
            const int count = __builtin_amdgcn_readfirstlane(jobs[j].count);
            b = w2 + ((int64_t)e * H + n0 + lr) * I + lg * 16;
            sb = s2 + ((int64_t)e * NB + (n0 >> 7)) * SP;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = start + min(16 * r + lr, count - 1);
                a[r] = 16 * r + lr < count ? (uint32_t)(row * I + lg * 16) : kNoRow;
                sa[r] = sh + (int64_t)row * SP;
            }
        };
        auto load = [&](Block<R, 1, kE8>& s) __attribute__((always_inline)) {
            load_chunks(b + lk * 128, s.b[0]);
            s.sb[0] = sb[lk];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                load_chunks(hbuf, a[r] + lk * 128, s.a[r]);
                s.sa[r] = sa[r][lk];
            }
            if (++lk == KB) {
                lk = 0;
                lj = min(lj + 1, n_jobs - 1);
                aim(lj);
            }
        };
        aim(lj);
#pragma unroll
        for (int d = 0; d < D; ++d) load(ring[d]);
        int j = first / KB, kb = first % KB;
        v4f acc[R][1];
        clear(acc);
        for (int s = first; s < last; s += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (s + d < last) {
                    const int rows = __builtin_amdgcn_readfirstlane(jobs[j].count);
                    multiply(ring[d], rows, acc);
                    if (++kb == KB || s + d + 1 == last) {
                        const int start = __builtin_amdgcn_readfirstlane(jobs[j].start);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const int i = 16 * r + lr;
                            if (i < rows) {
                                // two rows may be one token: LDS adds, in lane order
                                const float w = row_w[start + i];
                                float* const to = mine + row_t[start + i] * 16 + 4 * lg;
#pragma unroll
                                for (int q = 0; q < 4; ++q) atomicAdd(to + q, w * acc[r][0][q]);
                            }
                        }
                        clear(acc);
                        kb = 0;
                        ++j;
                    }
                }
                load(ring[d]);
            }
        }
    }
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

template <int R, bool kE8>
static dg_status moe_r(const MoeArgs& a, hipStream_t stream) {
    const MoeLayout at(a.T, a.k, a.E, a.H, a.I);
    uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
    MoeUnit* const units = reinterpret_cast<MoeUnit*>(ws + at.units);
    int32_t* const order = reinterpret_cast<int32_t*>(ws + at.order);
    int32_t* const place = reinterpret_cast<int32_t*>(ws + at.place);
    uint8_t* const codes = ws + at.codes;
    void* const scales = ws + at.scales;
    const int P = a.T * a.k, U = std::min(P, a.E);
    constexpr int D = R == 4 ? 3 : 4;
    hipLaunchKernelGGL((moe_gate_up_kernel<R, D, kE8>), dim3(a.I / 128, U), dim3(64 * kPanelWaves),
                       (panel_lds<R, 2, D>()) + P * 2, stream, a.x, a.sx, a.ids, a.w13, a.s13, units, order,
                       place, codes, scales,
                       P, a.k, a.E, a.H, a.I, P <= a.E);
    const dg_status s = launched();
    if (s != DG_OK) return s;
    if (a.T > kFusedTokens) {
        float* const out = reinterpret_cast<float*>(ws + at.out);
        constexpr int D2 = 3;
        hipLaunchKernelGGL((moe_down_rows_kernel<R, D2, kE8>), dim3(a.H / 128, U), dim3(64 * kPanelWaves),
                           (panel_lds<R, 1, D2>()), stream, codes, scales, a.w2, a.s2, units, out, P, a.H, a.I);
        if (launched() != DG_OK) return DG_ERR_HIP;
        hipLaunchKernelGGL(moe_combine_kernel, dim3((a.H + 1023) / 1024, a.T), dim3(256), 0, stream, out, a.ids,
                           place, a.weights, a.y, a.k, a.E, a.H);
        return launched();
    }
    constexpr int W = 4;
    const size_t lds = W * a.T * 64 + ((P + 3) & ~3) * 4 + (U + P / (16 * R)) * sizeof(MoeJob) + P * 2;
    hipLaunchKernelGGL((moe_down_kernel<R, kE8, W>), dim3(a.H / 16), dim3(64 * W), lds, stream, codes,
                       scales, a.weights, a.w2, a.s2, units, order, a.y, a.T, U, a.k, a.H, a.I);
    return launched();
}

template <bool kE8>
static dg_status moe_scales(const MoeArgs& a, hipStream_t stream) {
    if (a.T <= 16) return moe_r<1, kE8>(a, stream);
    if (a.T <= 32) return moe_r<2, kE8>(a, stream);
    return moe_r<4, kE8>(a, stream);
}

dg_status launch_moe(const MoeArgs& a, bool e8m0, hipStream_t stream) {
    return e8m0 ? moe_scales<true>(a, stream) : moe_scales<false>(a, stream);
}

}  // namespace dg
