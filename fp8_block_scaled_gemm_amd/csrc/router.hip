// Expert router: the k best experts of each token with their weights, and the
// gradient of those weights.  include/dg_ops.h has the definition.
//
// One wave handles one token.  Lane l holds the NV logits of experts
// [NV l, NV l + NV), so lane order is expert order and the first lane of a
// ballot is the lowest index.  A rank is compared as an unsigned integer that
// orders like the number: 32 bits of the logit itself, or 64 bits of the score
// plus bias.  The 64-bit rank keeps the choice of experts independent of how
// an fp32 exponential rounds; scores that become weights are fp32.
//
// Bound: a row is E loads and k dependent rounds of a wave-wide maximum, so for
// one row latency sets the time.  256 fp32 experts, 8 chosen in 4 of 8 groups by
// biased sigmoid: one row 5.4 us, 4096 rows 11.1 us, 9.8 in a sequence of calls
// (4.5 MB; 1, 2, 8 or 16 rows a workgroup instead of 4 take as long).  All 4096
// waves are resident at once, so what they take beyond one row's time is issue:
// 256 64-bit scores a row and rounds that cost a whole wave.  The gradient of
// 8192 x 128 bf16, softmax: 5.2 us for 4.7 MB.
#include "device_common.h"
#include "ops_launch.h"
#include "wave_ops.h"

#include <algorithm>
#include <cmath>

namespace dg {

constexpr double kTopkEps = 1e-20;  // added to the sum that weights are divided by
constexpr int kRowsPerBlock = 4;    // one wave each

template <class In>
__device__ __forceinline__ float to_float(In v) {
    if constexpr (sizeof(In) == 2)
        return __uint_as_float((uint32_t)v << 16);
    else
        return v;
}

// Unsigned integers ordered like the numbers (no NaN); -0 counts as +0, so
// that equal numbers tie.
__device__ __forceinline__ uint32_t order32(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order64(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// exp(x - top) with +infinity shared equally: the entries equal to an infinite
// maximum count 1 each, all others 0.
template <class F>
__device__ __forceinline__ F exp_below(F x, F top) {
    if (top == (F)INFINITY) return x == top ? (F)1 : (F)0;
    return exp(x - top);
}

// A lane's NV values of a row; one load where the rows keep it aligned.
template <class In, int NV>
__device__ __forceinline__ void load_row(const In* row, int E, int lane, float (&x)[NV]) {
    constexpr int kVec = NV * sizeof(In) > 16 ? 16 / sizeof(In) : NV;
    typedef In Vec __attribute__((ext_vector_type(kVec)));
    const int e0 = lane * NV;
    if (E % NV == 0) {
#pragma unroll
        for (int i = 0; i < NV; i += kVec) {
            if (e0 < E) {
                const Vec v = *reinterpret_cast<const Vec*>(row + e0 + i);
#pragma unroll
                for (int q = 0; q < kVec; ++q) x[i + q] = to_float((In)v[q]);
            } else {
#pragma unroll
                for (int q = 0; q < kVec; ++q) x[i + q] = -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = e0 + i < E ? to_float(row[e0 + i]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (!(x[i] > -INFINITY)) x[i] = -INFINITY;  // NaN is masked like -infinity
}

// The two largest of two pairs, each with first >= second.
struct Best2 {
    double first, second;
    __device__ __forceinline__ void take(double f, double s) {
        second = fmax(fmin(first, f), fmax(second, s));
        first = fmax(first, f);
    }
    template <int kCtrl>
    __device__ __forceinline__ void merge_lanes() {
        const double f = dpp_move<kCtrl, 0xf>(first, first), s = dpp_move<kCtrl, 0xf>(second, second);
        take(f, s);
    }
    // a group with one open expert is ranked by that one
    __device__ __forceinline__ double value() const {
        return second > -(double)INFINITY ? first + second : first;
    }
};

// Ranks of experts outside the topk_group best groups become -infinity (as
// every closed expert's is).  `lds` holds 64 max(NV, 2) doubles of the wave.
template <int NV>
__device__ __forceinline__ void close_groups(double (&r)[NV], double* lds, int E, int n_group,
                                             int topk_group, int lane) {
    const double none = -(double)INFINITY;
    const int size = E / n_group, lanes = size / NV;  // lanes of a group, where it is whole lanes
    Best2 best = {none, none};
    if (size % NV == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) best.take(r[i], none);
    }
    if (size % NV == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0) {
        // groups of 1 .. 16 lanes: merged by moves within rows of 16 lanes
        if (lanes >= 2) best.merge_lanes<0xb1>();   // swap neighbours
        if (lanes >= 4) best.merge_lanes<0x4e>();   // swap pairs
        if (lanes >= 8) best.merge_lanes<0x141>();  // mirror 8
        if (lanes >= 16) best.merge_lanes<0x140>(); // mirror 16
        const double mine = best.value();
        const int group = lane / lanes;
        const v2u bits = __builtin_bit_cast(v2u, mine);
        int before = 0;  // groups ahead of this lane's
        for (int g = 0; g < n_group; ++g) {
            const double o = __builtin_bit_cast(
                double, v2u{(uint32_t)__builtin_amdgcn_readlane((int)bits[0], g * lanes),
                            (uint32_t)__builtin_amdgcn_readlane((int)bits[1], g * lanes)});
            before += o > mine || (o == mine && g < group);
        }
        if (before >= topk_group) {
#pragma unroll
            for (int i = 0; i < NV; ++i) r[i] = none;
        }
        return;
    }
    // any other size: lane g gathers group g from LDS
    const bool pairs = NV >= 2 && size % NV == 0;  // the lanes' two best are enough
    if (pairs) {
        lds[lane] = best.first;
        lds[64 + lane] = best.second;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) lds[lane * NV + i] = r[i];
    }
    wave_sync();
    best = {none, none};
    if (lane < n_group) {
        const int n = pairs ? lanes : size;
        for (int i = lane * n; i < (lane + 1) * n; ++i) best.take(lds[i], pairs ? lds[64 + i] : none);
    }
    const double mine = best.value();
    const v2u bits = __builtin_bit_cast(v2u, mine);
    int before = 0;
    for (int g = 0; g < n_group; ++g) {
        const double o = __builtin_bit_cast(double, v2u{(uint32_t)__builtin_amdgcn_readlane((int)bits[0], g),
                                                        (uint32_t)__builtin_amdgcn_readlane((int)bits[1], g)});
        before += o > mine || (o == mine && g < lane);
    }
    const uint64_t open = __ballot(lane < n_group && before < topk_group);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        if (e >= E || !((open >> (e / size)) & 1)) r[i] = none;
    }
}

template <class In, int NV>
__global__ __launch_bounds__(64 * kRowsPerBlock) void topk_kernel(
    const In* __restrict__ logits, const float* __restrict__ bias, int32_t* __restrict__ ids,
    float* __restrict__ weights, int64_t T, int E, int k, int n_group, int topk_group, bool sigmoid,
    bool renormalize, float scale) {
    __shared__ double ranks[kRowsPerBlock][64 * (NV < 2 ? 2 : NV)];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRowsPerBlock + w;
    if (t >= T) return;
    float x[NV], b[NV];
    load_row<In, NV>(logits + t * E, E, lane, x);
#pragma unroll
    for (int i = 0; i < NV; ++i) b[i] = bias && lane * NV + i < E ? bias[lane * NV + i] : 0.0f;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
    top = wave_max(top);

    // ranks as ordered integers; 0 is below every open expert's
    uint64_t key[NV];
    if (bias == nullptr && n_group == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = x[i] > -INFINITY ? (uint64_t)order32(x[i]) << 32 : 0;
    } else {
        double r[NV];
        double sum = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            r[i] = x[i] == -INFINITY ? 0.0
                   : sigmoid         ? 1.0 / (1.0 + exp(-(double)x[i]))
                                     : exp_below<double>(x[i], top);
            sum += r[i];
        }
        if (!sigmoid) {
            sum = wave_sum(sum);
#pragma unroll
            for (int i = 0; i < NV; ++i) r[i] /= sum;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            r[i] += (double)b[i];
            if (!(x[i] > -INFINITY && r[i] > -(double)INFINITY)) r[i] = -(double)INFINITY;
        }
        if (n_group > 1) close_groups<NV>(r, ranks[w], E, n_group, topk_group, lane);
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = r[i] > -(double)INFINITY ? order64(r[i]) : 0;
    }

    // k rounds: the wave's largest rank, at its lowest index.  Ranks are told
    // apart by their upper halves (an open one's is never 0); only when those
    // tie do the lower halves decide, then the index.  The comparisons' lane
    // masks are scalars, so a round is about 20 vector instructions for 256
    // experts; with 64-bit comparisons and selects per lane it was 55.  (4096
    // rows of 256, 8 chosen in 4 of 8 groups: 12.6 -> 12.2 us, as what a round
    // waits for is the chain of its wave-wide maximum.)
    uint32_t hi[NV], lo[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        hi[i] = (uint32_t)(key[i] >> 32);
        lo[i] = (uint32_t)key[i];
    }
    int my_id = -1;
    for (int j = 0; j < k; ++j) {
        uint32_t most = hi[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) most = max(most, hi[i]);
        most = wave_max(most);
        if (most == 0) break;
        uint64_t mask[NV];
        int n = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            mask[i] = __ballot(hi[i] == most);
            n += __popcll(mask[i]);
        }
        if (n > 1) {
            uint32_t low = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) low = hi[i] == most ? max(low, lo[i]) : low;
            low = wave_max(low);
            uint64_t any = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                mask[i] = __ballot(hi[i] == most && lo[i] == low);
                any |= mask[i];
            }
            // the lowest lane, there the lowest slot
            uint64_t only = any & (0 - any);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                mask[i] &= only;
                only ^= mask[i];
            }
        }
        int id = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (mask[i]) id = __builtin_ctzll(mask[i]) * NV + i;
            if ((mask[i] >> lane) & 1) hi[i] = 0;
        }
        if (lane == j) my_id = id;
    }
    float my_x = my_id >= 0 ? to_float(logits[t * E + my_id]) : -INFINITY;

    float weight = 0;
    if (sigmoid) {
        // one score per lane: 64 bits cost nothing and keep scores that fp32
        // would flush apart before they are divided by their sum
        double p = my_id >= 0 ? 1.0 / (1.0 + exp(-(double)my_x)) : 0.0;
        if (renormalize) p /= wave_sum(p) + kTopkEps;
        weight = (float)p;
    } else {
        float sum = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += x[i] > -INFINITY ? exp_below<float>(x[i], top) : 0.0f;
        sum = wave_sum(sum);
        weight = my_id >= 0 ? exp_below<float>(my_x, top) / sum : 0.0f;
        if (renormalize) weight /= wave_sum(weight) + (float)kTopkEps;
    }
    if (lane < k) {
        ids[t * k + lane] = my_id;
        weights[t * k + lane] = weight * scale;
    }
}

template <class In>
__device__ __forceinline__ In from_float(float v) {
    if constexpr (sizeof(In) == 2)
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    else
        return v;
}

template <class In, int NV>
__device__ __forceinline__ void store_row(In* row, int E, int lane, const float (&v)[NV]) {
    constexpr int kVec = NV * sizeof(In) > 16 ? 16 / sizeof(In) : NV;
    typedef In Vec __attribute__((ext_vector_type(kVec)));
    const int e0 = lane * NV;
    if (E % NV == 0) {
        if (e0 >= E) return;
#pragma unroll
        for (int i = 0; i < NV; i += kVec) {
            Vec o;
#pragma unroll
            for (int q = 0; q < kVec; ++q) o[q] = from_float<In>(v[i + q]);
            *reinterpret_cast<Vec*>(row + e0 + i) = o;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (e0 + i < E) row[e0 + i] = from_float<In>(v[i]);
    }
}

template <class In, int NV>
__global__ __launch_bounds__(64 * kRowsPerBlock) void topk_backward_kernel(
    const In* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ grad_w,
    In* __restrict__ grad, int64_t T, int E, int k, bool sigmoid, bool renormalize, float scale) {
    __shared__ float dense[kRowsPerBlock][64 * NV];  // gradient of the row's scores
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRowsPerBlock + w;
    if (t >= T) return;
    const In* row = logits + t * E;
    float x[NV];
    load_row<In, NV>(row, E, lane, x);
    int id = lane < k ? ids[t * k + lane] : -1;
    if (id < 0 || id >= E) id = -1;
    float g = id >= 0 ? grad_w[t * k + lane] * scale : 0.0f;
    const float xs = id >= 0 ? to_float(row[id]) : -INFINITY;
    if (!(xs > -INFINITY)) {  // a masked expert's weight is 0 whatever its gradient
        id = -1;
        g = 0.0f;
    }
    float out[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) dense[w][lane + 64 * i] = 0.0f;
    wave_sync();
    if (sigmoid) {
        // only the listed experts have a gradient: one 64-bit score per lane
        const double p = id >= 0 ? 1.0 / (1.0 + exp(-(double)xs)) : 0.0;
        double d = g;
        if (renormalize) {
            // w_j = p_j / S: dL/dp_j = (g_j - sum_i g_i p_i / S) / S
            const double total = wave_sum(p) + kTopkEps;
            d = (d - wave_sum(d * p) / total) / total;
        }
        if (id >= 0) atomicAdd(&dense[w][id], (float)(d * p * (1.0 - p)));
        wave_sync();
#pragma unroll
        for (int i = 0; i < NV; ++i) out[i] = dense[w][lane * NV + i];
        store_row<In, NV>(grad + t * E, E, lane, out);
        return;
    }

    float top = -INFINITY, rsum = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
    top = wave_max(top);
    float e[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        e[i] = x[i] > -INFINITY ? exp_below<float>(x[i], top) : 0.0f;
        rsum += e[i];
    }
    rsum = wave_sum(rsum);
    rsum = rsum > 0.0f ? 1.0f / rsum : 0.0f;  // 0: no expert is open
    const float p = id >= 0 ? exp_below<float>(xs, top) * rsum : 0.0f;
    if (renormalize) {
        const float total = wave_sum(p) + (float)kTopkEps;
        const float mean = wave_sum(g * p) / total;
        g = id >= 0 ? (g - mean) / total : 0.0f;
    }
    const float dot = wave_sum(g * p);
    if (id >= 0) atomicAdd(&dense[w][id], g);
    wave_sync();
#pragma unroll
    for (int i = 0; i < NV; ++i)  // masked: 0, also where `dot` is not finite
        out[i] = x[i] > -INFINITY ? e[i] * rsum * (dense[w][lane * NV + i] - dot) : 0.0f;
    store_row<In, NV>(grad + t * E, E, lane, out);
}

static int64_t row_blocks(int64_t T) { return (T + kRowsPerBlock - 1) / kRowsPerBlock; }

// More rows than one grid holds (2^26 of 64 lanes) take several launches.
constexpr int64_t kMaxRows = int64_t(1) << 25;

template <class In, int NV>
static dg_status topk_nv(const TopkArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((topk_kernel<In, NV>), dim3((unsigned)row_blocks(a.T)), dim3(64 * kRowsPerBlock),
                       0, stream, static_cast<const In*>(a.logits), a.bias, a.ids, a.weights, a.T, a.E,
                       a.k, a.n_group, a.topk_group, a.sigmoid, a.renormalize, a.scale);
    return launched();
}

template <class In>
static dg_status topk_in(const TopkArgs& a, hipStream_t stream) {
    if (a.E <= 64) return topk_nv<In, 1>(a, stream);
    if (a.E <= 128) return topk_nv<In, 2>(a, stream);
    if (a.E <= 256) return topk_nv<In, 4>(a, stream);
    if (a.E <= 512) return topk_nv<In, 8>(a, stream);
    return topk_nv<In, 16>(a, stream);
}

dg_status launch_topk(const TopkArgs& a, bool bf16, hipStream_t stream) {
    if (row_blocks(a.T) > 0x7fffffff) return DG_ERR_SHAPE;
    for (int64_t t = 0; t < a.T; t += kMaxRows) {
        TopkArgs part = a;
        part.logits = static_cast<const char*>(a.logits) + t * a.E * (bf16 ? 2 : 4);
        part.ids = a.ids + t * a.k;
        part.weights = a.weights + t * a.k;
        part.T = std::min(a.T - t, kMaxRows);
        const dg_status s = bf16 ? topk_in<uint16_t>(part, stream) : topk_in<float>(part, stream);
        if (s != DG_OK) return s;
    }
    return DG_OK;
}

template <class In, int NV>
static dg_status backward_nv(const TopkBackwardArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((topk_backward_kernel<In, NV>), dim3((unsigned)row_blocks(a.T)),
                       dim3(64 * kRowsPerBlock), 0, stream, static_cast<const In*>(a.logits), a.ids,
                       a.grad_weights, static_cast<In*>(a.grad_logits), a.T, a.E, a.k, a.sigmoid,
                       a.renormalize, a.scale);
    return launched();
}

template <class In>
static dg_status backward_in(const TopkBackwardArgs& a, hipStream_t stream) {
    if (a.E <= 64) return backward_nv<In, 1>(a, stream);
    if (a.E <= 128) return backward_nv<In, 2>(a, stream);
    if (a.E <= 256) return backward_nv<In, 4>(a, stream);
    if (a.E <= 512) return backward_nv<In, 8>(a, stream);
    return backward_nv<In, 16>(a, stream);
}

dg_status launch_topk_backward(const TopkBackwardArgs& a, bool bf16, hipStream_t stream) {
    if (row_blocks(a.T) > 0x7fffffff) return DG_ERR_SHAPE;
    for (int64_t t = 0; t < a.T; t += kMaxRows) {
        TopkBackwardArgs part = a;
        part.logits = static_cast<const char*>(a.logits) + t * a.E * (bf16 ? 2 : 4);
        part.ids = a.ids + t * a.k;
        part.grad_weights = a.grad_weights + t * a.k;
        part.grad_logits = static_cast<char*>(a.grad_logits) + t * a.E * (bf16 ? 2 : 4);
        part.T = std::min(a.T - t, kMaxRows);
        const dg_status s = bf16 ? backward_in<uint16_t>(part, stream) : backward_in<float>(part, stream);
        if (s != DG_OK) return s;
    }
    return DG_OK;
}

}  // namespace dg
