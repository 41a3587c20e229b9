// 8-bit integer NT products for gfx950 (dense and contiguous-grouped), and the
// quantizer of their operands.  include/dg_int8.h has the definitions.
//
// The sum over K is exact in int32, so there is nothing to promote between K
// blocks: the matrix instruction accumulates straight into the tile's
// registers, and the scales are applied once, in the epilogue.
#include "experts_launch.h"

#include <type_traits>

#include "rows_common.h"
#include "tiles.h"

namespace dg {

typedef int v4i __attribute__((ext_vector_type(4)));

// Tiles, K slabs, stages and barriers are those of the FP8 products' kernel: a
// K block of 128 bytes a row, two stages of A and B in LDS, chunk c of row r at
// c ^ (r & 7), lane (lr, lg) of a fragment read taking chunks lg and lg + 4 of
// row lr.  Each of the two chunks is one operand of v_mfma_i32_16x16x64_i8 (K
// [16 g, 16 g + 16) of lane group g): which 64 of the block's 128 values an
// instruction takes is free, as A and B agree.  B goes first, so that a lane
// owns one output row and four consecutive columns of a sub-tile.
template <class T, bool kGrouped, bool kMixed = false>
__global__ __launch_bounds__(T::kThreads, 2) void int8_gemm_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ sa, const uint8_t* __restrict__ B,
    const float* __restrict__ sb, uint16_t* __restrict__ D, const int32_t* __restrict__ layout, int64_t rows, int64_t N,
    int64_t K, int64_t G, int m_blocks, int n_blocks) {
    __shared__ __align__(1024) uint8_t smem[T::kSmem];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int KB = (int)(K >> 7);
    const int lr = lane & 15, lg = lane >> 4;
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
    const int wcol = wn * T::WN;

    TileInfo ti;
    ti.ok0 = ti.ok1 = 0;
    ti.g = 0;
    if constexpr (kMixed) {
        // the 128-row block blockIdx.x, from its second largest valid id on
        ti.m0 = blockIdx.x * T::BM;
        ti.n0 = 0;
        ti.valid = T::BM;
        ti.arow0 = ti.m0;
        if (!block_group(layout, G, (int)G, lane, ti) || !block_group(layout, G, ti.g, lane, ti)) return;
    } else {
        const int tile = xcd_tile(blockIdx.x, m_blocks * n_blocks);
        if (tile < 0) return;
        const int span = T::kGroupM * n_blocks;
        const int first_m = (tile / span) * T::kGroupM;
        const int gm = min(m_blocks - first_m, T::kGroupM);
        const int in_span = tile % span;
        ti.m0 = (first_m + in_span % gm) * T::BM;
        ti.n0 = (in_span / gm) * T::BN;
        ti.arow0 = ti.m0;
        if constexpr (kGrouped) {
            static_assert(!kGrouped || T::BM == 128, "one group per 128-row block");
            if (!block_group(layout, G, (int)G, lane, ti)) return;
            ti.valid = T::BM;
        } else {
            ti.valid = (int)min<int64_t>(T::BM, rows - ti.m0);
        }
    }

    for (;;) {
        uint8_t* const smA = smem;
        uint8_t* const smB = smem + 2 * T::kStageA;
        const int sub = lane >> 3, lchunk = (lane & 7) ^ sub;
        const uint32_t offRow = (uint32_t)(wave * 8 + sub) * (uint32_t)K + lchunk * 16;
        const int vn = (int)min<int64_t>(T::BN, N - ti.n0);
        const uint8_t* tileA = A + ti.arow0 * K;
        const uint8_t* tileB = B + ((int64_t)ti.g * N + ti.n0) * K;
        // loads [i0, i1) of this wave's share of the A slab of block kb; blocks
        // past the last one get an empty buffer, and so count like the others
        auto issue_a = [&](int kb, int st, int i0, int i1) __attribute__((always_inline)) {
            const v4u rs = buffer_rsrc(tileA + kb * 128, kb < KB ? (uint32_t)ti.valid * (uint32_t)K - kb * 128 : 0u);
#pragma unroll
            for (int i = i0; i < i1; ++i)
                load_lds_16(rs, offRow + (uint32_t)(i * T::kWaves * 8) * (uint32_t)K,
                            smA + st * T::kStageA + (wave + i * T::kWaves) * 1024);
        };
        auto issue_b = [&](int kb, int st) __attribute__((always_inline)) {
            const v4u rs = buffer_rsrc(tileB + kb * 128, kb < KB ? (uint32_t)vn * (uint32_t)K - kb * 128 : 0u);
#pragma unroll
            for (int i = 0; i < T::kLoadsB; ++i) {
                if ((T::BN / 8) % T::kWaves != 0 && wave + i * T::kWaves >= T::BN / 8) break;
                load_lds_16(rs, offRow + (uint32_t)(i * T::kWaves * 8) * (uint32_t)K,
                            smB + st * T::kStageB + (wave + i * T::kWaves) * 1024);
            }
        };
        constexpr int kRowStep = 16 * T::WAVES_M;
        const int chunk_lo = (lg ^ (lr & 7)) << 4, chunk_hi = chunk_lo ^ 64;
        const int fragA = (16 * wm + lr) * 128, fragB = (wcol + lr) * 128;

        v4i acc[T::TM][T::TN];
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
#pragma unroll
            for (int j = 0; j < T::TN; ++j) acc[i][j] = v4i{0, 0, 0, 0};
        v4i b[T::TN][2];
        auto mma_rows = [&](int st, int i0, int i1) __attribute__((always_inline)) {
            const uint8_t* stA = smA + st * T::kStageA + fragA;
#pragma unroll
            for (int i = i0; i < i1; ++i) {
                const v4i a0 = *reinterpret_cast<const v4i*>(stA + i * kRowStep * 128 + chunk_lo);
                const v4i a1 = *reinterpret_cast<const v4i*>(stA + i * kRowStep * 128 + chunk_hi);
#pragma unroll
                for (int j = 0; j < T::TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j][0], a0, acc[i][j], 0, 0, 0);
#pragma unroll
                for (int j = 0; j < T::TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j][1], a1, acc[i][j], 0, 0, 0);
            }
        };
        constexpr int kAfter = T::kLoadsA + T::kLoadsBMin;
        static_assert(T::kLoadsA % 2 == 0 && kAfter < 64, "A slab halves, vmcnt range");
        // One K block in two halves, two barriers: a slab's buffer is loaded
        // again (block kb + 2) as soon as the barrier that frees it has passed,
        // so that every load has one and a half blocks to land.
        auto step = [&](int kb, int st) __attribute__((always_inline)) {
            const uint8_t* stB = smB + st * T::kStageB + fragB;
#pragma unroll
            for (int j = 0; j < T::TN; ++j) {
                b[j][0] = *reinterpret_cast<const v4i*>(stB + j * 2048 + chunk_lo);
                b[j][1] = *reinterpret_cast<const v4i*>(stB + j * 2048 + chunk_hi);
            }
            mma_rows(st, 0, T::TM / 2);
            wait_vmcnt_lgkm0<kAfter>();  // A rows [BM/2, BM) of kb
            lds_barrier();
            issue_a(kb + 2, st, 0, T::kLoadsA / 2);
            issue_b(kb + 2, st);
            mma_rows(st, T::TM / 2, T::TM);
            wait_vmcnt_lgkm0<kAfter>();  // A rows [0, BM/2) and B of kb+1
            lds_barrier();
            issue_a(kb + 2, st, T::kLoadsA / 2, T::kLoadsA);
        };
        issue_a(0, 0, 0, T::kLoadsA);
        issue_b(0, 0);
        issue_a(1, 1, 0, T::kLoadsA / 2);
        issue_b(1, 1);
        wait_vmcnt<0>();
        lds_barrier();
        issue_a(1, 1, T::kLoadsA / 2, T::kLoadsA);
        for (int kb = 0; kb < KB; kb += 2) {
            step(kb, 0);
            if (kb + 1 < KB) step(kb + 1, 1);
        }
        wait_vmcnt<0>();  // the empty loads of the last steps have retired
        lds_barrier();

        // epilogue: scales by row and column, rounding, and out through LDS
        v4f col_scale[T::TN];
#pragma unroll
        for (int j = 0; j < T::TN; ++j) {
            const int64_t col = min<int64_t>(ti.n0 + wcol + 16 * j + 4 * lg, N - 4);
            col_scale[j] = *reinterpret_cast<const v4f*>(sb + (int64_t)ti.g * N + col);
        }
#pragma unroll
        for (int i = 0; i < T::TM; ++i) {
            const int row = 16 * (T::WAVES_M * i + wm) + lr;
            const float row_scale = sa[ti.arow0 + min(row, ti.valid - 1)];
#pragma unroll
            for (int j = 0; j < T::TN; ++j) {
                v4f v;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = (row_scale * col_scale[j][q]) * (float)acc[i][j][q];
                stage_bf16<T>(smem, row, wcol + 16 * j + 4 * lg, v);
            }
        }
        __syncthreads();
        store_staged<T, kGrouped>(smem, tid, ti, D, N);
        if constexpr (!kMixed) {
            break;
        } else {
            if ((int64_t)ti.n0 + T::BN < N) {
                ti.n0 += T::BN;
            } else {
                ti.n0 = 0;
                if (!block_group(layout, G, ti.g, lane, ti)) break;
            }
            lds_barrier();  // the staged tile has been stored before the next pass loads
        }
    }
}

template <class T, bool kGrouped>
static dg_status launch_tiled(const Int8Args& a, hipStream_t stream) {
    const int64_t m_blocks = (a.rows + T::BM - 1) / T::BM, n_blocks = (a.N + T::BN - 1) / T::BN;
    const int64_t grid = (m_blocks * n_blocks + kNumXcds - 1) / kNumXcds * kNumXcds;
    if (!grid_fits(grid, T::kThreads)) return DG_ERR_SHAPE;
    // per-lane 32-bit offsets into a tile's rows of K bytes: K < 2^17
    const auto* A = reinterpret_cast<const uint8_t*>(a.A);
    const auto* B = reinterpret_cast<const uint8_t*>(a.B);
    hipLaunchKernelGGL((int8_gemm_kernel<T, kGrouped>), dim3((unsigned)grid), dim3(T::kThreads), 0, stream, A, a.sa, B,
                       a.sb, a.D, a.layout, a.rows, a.N, a.K, a.G, (int)m_blocks, (int)n_blocks);
    if constexpr (kGrouped) {
        // blocks that carry more than one valid id
        if (launched() != DG_OK) return DG_ERR_HIP;
        hipLaunchKernelGGL((int8_gemm_kernel<T, true, true>), dim3((unsigned)m_blocks), dim3(T::kThreads), 0, stream, A,
                           a.sa, B, a.sb, a.D, a.layout, a.rows, a.N, a.K, a.G, (int)m_blocks, (int)n_blocks);
    }
    return launched();
}

using Int8Large = TileConfig<256, 256, 4, 2, 4>;
using Int8Rows128 = TileConfig<128, 256, 2, 4, 8>;
using Int8Narrow = TileConfig<128, 32, 2, 2, 8>;

dg_status launch_int8_gemm(const Int8Args& a, hipStream_t stream) {
    if (a.layout != nullptr) return launch_tiled<Int8Rows128, true>(a, stream);
    const int64_t large = ((a.rows + 255) / 256) * ((a.N + 255) / 256);
    if (2 * large <= device_cus()) return launch_tiled<Int8Narrow, false>(a, stream);
    return launch_tiled<Int8Large, false>(a, stream);
}

// One workgroup per row, read twice (the second time from its cache): the
// scale needs all of it.
template <bool kBf16>
__global__ __launch_bounds__(256) void quantize_int8_kernel(const void* __restrict__ x, int64_t K,
                                                            uint8_t* __restrict__ q, float* __restrict__ s) {
    __shared__ uint32_t tops[4];
    const int64_t m = blockIdx.x;
    const int tid = threadIdx.x;
    auto load = [&](int64_t c, float (&f)[8]) __attribute__((always_inline)) {
        if constexpr (kBf16) {
            unpack_bf16(*reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(x) + m * K + c * 8), f);
        } else {
            const v4f* const p = reinterpret_cast<const v4f*>(static_cast<const float*>(x) + m * K + c * 8);
            const v4f lo = p[0], hi = p[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = lo[e];
                f[4 + e] = hi[e];
            }
        }
    };
    uint32_t top = 0;
    for (int64_t c = tid; c < K / 8; c += 256) {
        float f[8];
        load(c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, magnitude_bits(f[e]));
    }
    const Int8Row row(block_max<4>(top, tops, tid));
    for (int64_t c = tid; c < K / 8; c += 256) {
        float f[8];
        load(c, f);
        *reinterpret_cast<v2u*>(q + m * K + c * 8) = row.codes(f);
    }
    if (tid == 0) s[m] = row.scale;
}

dg_status launch_quantize_int8(const void* x, bool bf16, int64_t M, int64_t K, int8_t* q, float* s, hipStream_t stream) {
    if (!grid_fits(M, 256)) return DG_ERR_SHAPE;
    auto* const codes = reinterpret_cast<uint8_t*>(q);
    if (bf16)
        hipLaunchKernelGGL(quantize_int8_kernel<true>, dim3((unsigned)M), dim3(256), 0, stream, x, K, codes, s);
    else
        hipLaunchKernelGGL(quantize_int8_kernel<false>, dim3((unsigned)M), dim3(256), 0, stream, x, K, codes, s);
    return launched();
}

}  // namespace dg
