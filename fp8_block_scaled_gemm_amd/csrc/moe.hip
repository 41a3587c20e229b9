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

namespace dg {

struct MoeUnit {
    int e, start, count, pad;
};

// Up to 16 R rows of one unit.
struct MoeJob {
    int e;
    uint16_t start, count;
};

// Workspace layout, in bytes from its start.
struct MoeLayout {
    int64_t units, order, hidden, codes, scales, total;
    MoeLayout(int64_t T, int64_t k, int64_t E, int64_t I) {
        const int64_t P = T * k, U = std::min(P, E);
        auto up = [](int64_t v) { return (v + 255) & ~int64_t(255); };
        units = 0;
        order = units + up(U * sizeof(MoeUnit));
        hidden = order + up(P * 4);
        codes = hidden + up(P * I * 4);
        scales = codes + up(P * I);
        total = scales + up(P * ((I / 128 + 3) & ~int64_t(3)) * 4);
    }
};

// Rows of one unit, found by each wave for itself from the ids: the pairs of
// the unit's expert in order, into `list` if given.  count is 0 when the unit
// has no expert here, or (units numbered by pair) an earlier pair named it.
__device__ __forceinline__ MoeUnit find_unit(const int32_t* __restrict__ ids, int P, int E, int unit,
                                             bool by_pair, int lane, uint16_t* list) {
    MoeUnit u;
    u.e = by_pair ? ids[unit] : unit;
    u.start = u.count = u.pad = 0;
    if (u.e < 0 || u.e >= E) return u;
    for (int base = 0; base < P; base += 64) {
        const int q = base + lane;
        const int id = q < P ? ids[q] : -1;
        const uint64_t same = __ballot(id == u.e);
        u.start += __popcll(__ballot(id >= 0 && id < u.e));
        if (by_pair && u.count == 0 && same != 0 && base + __builtin_ctzll(same) < unit) return u;
        if (list && id == u.e)
            list[u.count + __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                                     __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0))] =
                (uint16_t)q;
        u.count += __popcll(same);
    }
    return u;
}

// First product: hidden[row] = silu(gate) * up, fp32.  A workgroup's four
// waves take 16 hidden columns each of one unit; a wave multiplies the gate
// and the up rows of the weights by the same activations.
template <int R, bool kE8>
__global__ __launch_bounds__(256) void moe_gate_up_kernel(
    const uint8_t* __restrict__ x, const void* __restrict__ sx_v, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ w13, const void* __restrict__ s13_v, MoeUnit* __restrict__ units,
    int32_t* __restrict__ order, float* __restrict__ hidden, int P, int k, int E, int H, int I,
    bool by_pair) {
    using S = typename std::conditional<kE8, uint8_t, float>::type;
    const S* sx = static_cast<const S*>(sx_v);
    const S* s13 = static_cast<const S*>(s13_v);
    extern __shared__ __align__(16) uint8_t smem[];
    uint16_t* list = reinterpret_cast<uint16_t*>(smem);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const MoeUnit u = find_unit(ids, P, E, blockIdx.y, by_pair, lane, wave == 0 ? list : nullptr);
    if (blockIdx.x == 0 && threadIdx.x == 0) units[blockIdx.y] = u;
    if (u.count == 0) return;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < u.count; i += 256) order[u.start + i] = list[i];

    const int KB = H >> 7, SP = scale_pitch<kE8>(KB), n0 = (blockIdx.x * 4 + wave) * 16;
    const int NB = (2 * I + 127) >> 7;
    const uint8_t* b[2];
    const S* sb[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        b[c] = w13 + ((int64_t)u.e * 2 * I + c * I + n0 + lr) * H + lg * 16;
        sb[c] = s13 + ((int64_t)u.e * NB + ((c * I + n0) >> 7)) * SP;
    }
    for (int m0 = 0; m0 < u.count; m0 += 16 * R) {
        const int rows = u.count - m0;
        const uint8_t* a[R];
        const S* sa[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = list[min(m0 + 16 * r + lr, u.count - 1)] / k;
            a[r] = x + (int64_t)t * H + lg * 16;
            sa[r] = sx + (int64_t)t * SP;
        }
        v4f acc[R][2];
        clear(acc);
        constexpr int D = R == 1 ? 4 : 2;
        Block<R, 2, kE8> ring[D];
        auto load = [&](int kb, Block<R, 2, kE8>& s) __attribute__((always_inline)) {
            kb = min(kb, KB - 1);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                load_chunks(b[c] + kb * 128, s.b[c]);
                s.sb[c] = sb[c][kb];
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                load_chunks(a[r] + kb * 128, s.a[r]);
                s.sa[r] = sa[r][kb];
            }
        };
#pragma unroll
        for (int d = 0; d < D; ++d) load(d, ring[d]);
        for (int kb = 0; kb < KB; kb += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (kb + d < KB) multiply(ring[d], rows, acc);
                load(kb + d + D, ring[d]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = m0 + 16 * r + lr;
            if (row >= u.count) continue;
            v4f h;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float g = acc[r][0][q];
                h[q] = g / (1.0f + expf(-g)) * acc[r][1][q];
            }
            *reinterpret_cast<v4f*>(hidden + (int64_t)(u.start + row) * I + n0 + 4 * lg) = h;
        }
    }
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
        const uint8_t *b, *a[R];
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
                a[r] = codes + (int64_t)row * I + lg * 16;
                sa[r] = sh + (int64_t)row * SP;
            }
        };
        auto load = [&](Block<R, 1, kE8>& s) __attribute__((always_inline)) {
            load_chunks(b + lk * 128, s.b[0]);
            s.sb[0] = sb[lk];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                load_chunks(a[r] + lk * 128, s.a[r]);
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
    return MoeLayout(T, k, E, I).total;
}

template <int R, bool kE8>
static dg_status moe_r(const MoeArgs& a, hipStream_t stream) {
    const MoeLayout at(a.T, a.k, a.E, a.I);
    uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
    MoeUnit* const units = reinterpret_cast<MoeUnit*>(ws + at.units);
    int32_t* const order = reinterpret_cast<int32_t*>(ws + at.order);
    float* const hidden = reinterpret_cast<float*>(ws + at.hidden);
    uint8_t* const codes = ws + at.codes;
    void* const scales = ws + at.scales;
    const int P = a.T * a.k, U = std::min(P, a.E);
    hipLaunchKernelGGL((moe_gate_up_kernel<R, kE8>), dim3(a.I / 64, U), dim3(256), (P * 2 + 15) & ~15,
                       stream, a.x, a.sx, a.ids, a.w13, a.s13, units, order, hidden, P, a.k, a.E, a.H,
                       a.I, P <= a.E);
    dg_status s = launched();
    if (s != DG_OK) return s;
    s = kE8 ? launch_quantize_per_token_e8m0(hidden, P, a.I, codes, static_cast<uint8_t*>(scales), stream)
            : launch_quantize_per_token(hidden, P, a.I, codes, static_cast<float*>(scales), stream);
    if (s != DG_OK) return s;
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
