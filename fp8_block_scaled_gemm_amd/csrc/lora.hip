// A shared projection with each row's own low-rank adapter: the first small
// product here, the second in the epilogue of the dense GEMM (gemm.hip).
// include/dg_ops.h has the definition.
#include "ops_launch.h"

#include <algorithm>

#include "device_common.h"

namespace dg {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kShrinkWaves = 4;

// low[part][m][0..R) = scaling[a] * x_m lora_a[a]^T over the part's share of K,
// for the rows m that have an adapter.  A workgroup takes 16 rows, the distinct
// adapters number blockIdx.y, + gridDim.y, .. among them, and one part of K,
// which its waves split; the waves' sums meet in LDS.  Every lane holds row
// (lane & 15) of x; a product row belongs to one x row only, so rows of other
// adapters are computed beside it and dropped.
template <int RT>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ lora_a,
    const int32_t* __restrict__ ids, const float* __restrict__ scaling, float* __restrict__ low,
    int64_t M, int64_t K, int L, int R) {
    __shared__ float part[kShrinkWaves][16][16 * RT + 4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * 16, row = std::min(m0 + lr, M - 1);
    int id = m0 + lr < M ? ids[row] : -1;
    if (id < 0 || id >= L) id = -1;
    // the first row of each distinct adapter
    bool first = id >= 0;
    for (int d = 0; d < 15; ++d) {
        const int o = __shfl(id, d, 64);
        if (d < lr && o == id) first = false;
    }
    uint32_t leaders = (uint32_t)__ballot(first) & 0xffffu;
    const int steps = (int)(K >> 6), shares = gridDim.z * kShrinkWaves;
    const int share = blockIdx.z * kShrinkWaves + wave;
    const int s0 = (int)((int64_t)share * steps / shares), s1 = (int)((int64_t)(share + 1) * steps / shares);
    const uint16_t* const px = x + row * K + 8 * lg;
    for (int n = 0; leaders != 0; ++n, leaders &= leaders - 1) {
        if (n % gridDim.y != blockIdx.y) continue;
        const int a = __builtin_amdgcn_readfirstlane(__shfl(id, __builtin_ctz(leaders), 64));
        v4f acc[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
        const uint16_t* pa[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            pa[r] = lora_a + ((int64_t)a * R + std::min(16 * r + lr, R - 1)) * K + 8 * lg;
        for (int s = s0; s < s1; ++s) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = (int64_t)s * 64 + 32 * h;
                const v8bf xv = *reinterpret_cast<const v8bf*>(px + at);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        *reinterpret_cast<const v8bf*>(pa[r] + at), xv, acc[r], 0, 0, 0);
            }
        }
        __syncthreads();  // the last adapter's sums have been read
#pragma unroll
        for (int r = 0; r < RT; ++r) *reinterpret_cast<v4f*>(&part[wave][lr][16 * r + 4 * lg]) = acc[r];
        __syncthreads();
        const float scale = scaling[a];
        for (int i = threadIdx.x; i < 16 * R; i += 64 * kShrinkWaves) {
            const int mi = i / R, r = i - mi * R;
            float sum = 0;
#pragma unroll
            for (int w = 0; w < kShrinkWaves; ++w) sum += part[w][mi][r];
            if (__shfl(id, mi, 64) == a) low[((int64_t)blockIdx.z * M + m0 + mi) * R + r] = scale * sum;
        }
    }
}

// Parts of K: a few rows give few workgroups, so K is split over more of them.
static int shrink_parts(int64_t M, int64_t K) {
    const int64_t blocks = (M + 15) / 16, most = std::max<int64_t>(1, K / 512);
    return (int)std::min(std::max<int64_t>(1, 64 / blocks), most);
}

int64_t lora_workspace(int64_t M, int64_t N, int64_t K, int64_t R) {
    return shrink_parts(M, K) * M * R * 4;
}

template <int RT>
static void shrink(const LoraArgs& a, float* low, int parts, hipStream_t stream) {
    const int64_t blocks = (a.M + 15) / 16;
    const int slots = (int)std::min<int64_t>(a.L, blocks >= 64 ? 4 : 16);
    hipLaunchKernelGGL((lora_shrink_kernel<RT>), dim3((unsigned)blocks, slots, parts),
                       dim3(64 * kShrinkWaves), 0, stream, a.x, a.lora_a, a.ids, a.scaling, low, a.M,
                       a.K, a.L, a.R);
}

dg_status launch_lora(const LoraArgs& a, bool e8m0, hipStream_t stream) {
    const int parts = shrink_parts(a.M, a.K);
    float* const low = static_cast<float*>(a.workspace);
    if (a.R <= 16)
        shrink<1>(a, low, parts, stream);
    else if (a.R <= 32)
        shrink<2>(a, low, parts, stream);
    else if (a.R <= 64)
        shrink<4>(a, low, parts, stream);
    else
        shrink<8>(a, low, parts, stream);
    const dg_status s = launched();
    if (s != DG_OK) return s;
    GemmArgs g{a.A, a.sa, a.B, a.sb, a.D, nullptr, a.M, a.N, a.K, 1, nullptr};
    g.e8m0 = e8m0;
    g.lora = LoraTail{low, a.lora_b, a.ids, parts, a.L, a.R};
    return launch_gemm(Form::DenseLora, g, stream);
}

}  // namespace dg
