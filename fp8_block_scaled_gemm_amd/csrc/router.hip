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
// Bound: a row is E loads and k dependent rounds of a wave-wide maximum, so
// latency, not bandwidth, sets the time (4096 x 256 fp32 is 4 MB).
#include "device_common.h"
#include "ops_launch.h"

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

// LDS written by some lanes of a wave before this is read by others after it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <class T, class F>
__device__ __forceinline__ T wave_reduce(T v, F f) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = f(v, __shfl_xor(v, d, 64));
    return v;
}

// exp(x - top) with +infinity shared equally: the entries equal to an infinite
// maximum count 1 each, all others 0.
template <class F>
__device__ __forceinline__ F exp_below(F x, F top) {
    if (top == (F)INFINITY) return x == top ? (F)1 : (F)0;
    return exp(x - top);
}

template <class In, int NV>
__device__ __forceinline__ void load_row(const In* row, int E, int lane, float (&x)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        x[i] = e < E ? to_float(row[e]) : -INFINITY;
        if (!(x[i] > -INFINITY)) x[i] = -INFINITY;  // NaN is masked like -infinity
    }
}

template <class In, int NV>
__global__ __launch_bounds__(64 * kRowsPerBlock) void topk_kernel(
    const In* __restrict__ logits, const float* __restrict__ bias, int32_t* __restrict__ ids,
    float* __restrict__ weights, int64_t T, int E, int k, int n_group, int topk_group, bool sigmoid,
    bool renormalize, float scale) {
    __shared__ uint64_t ranks[kRowsPerBlock][64 * NV];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRowsPerBlock + w;
    if (t >= T) return;
    float x[NV];
    load_row<In, NV>(logits + t * E, E, lane, x);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
    top = wave_reduce(top, [](float a, float b) { return fmaxf(a, b); });

    // ranks; 0 is below every open expert's
    uint64_t key[NV];
    if (bias == nullptr && n_group == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = x[i] > -INFINITY ? (uint64_t)order32(x[i]) << 32 : 0;
    } else {
        double p[NV];
        double sum = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            p[i] = x[i] == -INFINITY ? 0.0
                   : sigmoid         ? 1.0 / (1.0 + exp(-(double)x[i]))
                                     : exp_below<double>(x[i], top);
            sum += p[i];
        }
        if (!sigmoid) {
            sum = wave_reduce(sum, [](double a, double b) { return a + b; });
#pragma unroll
            for (int i = 0; i < NV; ++i) p[i] /= sum;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane * NV + i;
            if (bias && e < E) p[i] += (double)bias[e];
            key[i] = x[i] > -INFINITY && p[i] > -(double)INFINITY ? order64(p[i]) : 0;
        }
        if (n_group > 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i) ranks[w][lane * NV + i] = key[i];
            wave_sync();
            const int size = E / n_group;
            // lane g: the value of group g
            uint64_t value = 0;
            if (lane < n_group) {
                uint64_t first = 0, second = 0;
                for (int i = 0; i < size; ++i) {
                    const uint64_t r = ranks[w][lane * size + i];
                    if (r > first) {
                        second = first;
                        first = r;
                    } else if (r > second) {
                        second = r;
                    }
                }
                auto number = [](uint64_t r) {
                    return __longlong_as_double((long long)((r >> 63) ? r & ~0x8000000000000000ull : ~r));
                };
                if (first) value = order64(number(first) + (second ? number(second) : 0.0));
            }
            // how many groups come before this one
            int before = 0;
            for (int g = 0; g < n_group; ++g) {
                const uint64_t o = __shfl(value, g, 64);
                before += o > value || (o == value && g < lane);
            }
            const uint64_t open = __ballot(lane < n_group && before < topk_group);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = lane * NV + i;
                if (e >= E || !((open >> (e / size)) & 1)) key[i] = 0;
            }
        }
    }

    // k rounds: the wave's largest rank, at its lowest index
    int my_id = -1;
    float my_x = -INFINITY;
    for (int j = 0; j < k; ++j) {
        uint64_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NV; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint64_t m = wave_reduce(best, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
        if (m == 0) break;
        const int owner = __builtin_ctzll(__ballot(best == m));
        const int slot = __shfl(at, owner, 64);
        float v = x[0];
#pragma unroll
        for (int i = 1; i < NV; ++i)
            if (slot == i) v = x[i];
        v = __shfl(v, owner, 64);
        if (lane == j) {
            my_id = owner * NV + slot;
            my_x = v;
        }
        if (lane == owner) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (slot == i) key[i] = 0;
        }
    }

    auto add = [](auto a, auto b) { return a + b; };
    float weight = 0;
    if (sigmoid) {
        // one score per lane: 64 bits cost nothing and keep scores that fp32
        // would flush apart before they are divided by their sum
        double p = my_id >= 0 ? 1.0 / (1.0 + exp(-(double)my_x)) : 0.0;
        if (renormalize) p /= wave_reduce(p, add) + kTopkEps;
        weight = (float)p;
    } else {
        float sum = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += x[i] > -INFINITY ? exp_below<float>(x[i], top) : 0.0f;
        sum = wave_reduce(sum, add);
        weight = my_id >= 0 ? exp_below<float>(my_x, top) / sum : 0.0f;
        if (renormalize) weight /= wave_reduce(weight, add) + (float)kTopkEps;
    }
    if (lane < k) {
        ids[t * k + lane] = my_id;
        weights[t * k + lane] = weight * scale;
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
    float xs = id >= 0 ? to_float(row[id]) : -INFINITY;
    if (!(xs > -INFINITY)) xs = -INFINITY;
    auto store_grad = [&](int e, float d) {
        if (e >= E) return;
        if constexpr (sizeof(In) == 2)
            grad[t * E + e] = __builtin_bit_cast(uint16_t, (__bf16)d);
        else
            grad[t * E + e] = d;
    };
    auto add = [](auto a, auto b) { return a + b; };
#pragma unroll
    for (int i = 0; i < NV; ++i) dense[w][lane + 64 * i] = 0.0f;
    wave_sync();
    if (sigmoid) {
        // only the listed experts have a gradient: one 64-bit score per lane
        const double p = id >= 0 ? 1.0 / (1.0 + exp(-(double)xs)) : 0.0;
        double d = g;
        if (renormalize) {
            // w_j = p_j / S: dL/dp_j = (g_j - sum_i g_i p_i / S) / S
            const double total = wave_reduce(p, add) + kTopkEps;
            d = (d - wave_reduce(d * p, add) / total) / total;
        }
        if (id >= 0) atomicAdd(&dense[w][id], (float)(d * p * (1.0 - p)));
        wave_sync();
#pragma unroll
        for (int i = 0; i < NV; ++i) store_grad(lane * NV + i, dense[w][lane * NV + i]);
        return;
    }

    float top = -INFINITY, rsum = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
    top = wave_reduce(top, [](float a, float b) { return fmaxf(a, b); });
    float e[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        e[i] = x[i] > -INFINITY ? exp_below<float>(x[i], top) : 0.0f;
        rsum += e[i];
    }
    rsum = wave_reduce(rsum, add);
    rsum = rsum > 0.0f ? 1.0f / rsum : 0.0f;  // 0: no expert is open
    const float p = id >= 0 && xs > -INFINITY ? exp_below<float>(xs, top) * rsum : 0.0f;
    if (renormalize) {
        const float total = wave_reduce(p, add) + (float)kTopkEps;
        const float mean = wave_reduce(g * p, add) / total;
        g = id >= 0 ? (g - mean) / total : 0.0f;
    }
    const float dot = wave_reduce(g * p, add);
    if (id >= 0) atomicAdd(&dense[w][id], g);
    wave_sync();
#pragma unroll
    for (int i = 0; i < NV; ++i)
        store_grad(lane * NV + i, e[i] * rsum * (dense[w][lane * NV + i] - dot));
}

static int64_t row_blocks(int64_t T) { return (T + kRowsPerBlock - 1) / kRowsPerBlock; }

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
    return bf16 ? topk_in<uint16_t>(a, stream) : topk_in<float>(a, stream);
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
    return bf16 ? backward_in<uint16_t>(a, stream) : backward_in<float>(a, stream);
}

}  // namespace dg
