// 8-bit integer NT products for gfx950 (dense and contiguous-grouped), and the
// quantizer of their operands.  include/dg_int8.h has the definitions.
//
// The sum over K is exact in int32, so there is nothing to promote between K
// blocks: the matrix instruction accumulates straight into the tile's
// registers, and the scales are applied once, in the epilogue.
#include "experts_launch.h"

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "rows_common.h"
#include "tiles.h"

namespace dg {

typedef int v4i __attribute__((ext_vector_type(4)));

// The tile kernel.  Four waves, one to a SIMD, as 2 x 2 over a BM x BN tile, so
// that a wave may hold 512 registers: 128 x 128 sums of a 256 x 256 tile, and
// two sets of fragments.  A K block is 128 bytes a row, loaded straight from
// memory into one of S stages of LDS, 16-byte chunk c of row r at c ^ (r & 7).
// Lane (lr, lg) of a fragment read takes chunk lg (the block's first half) or
// lg + 4 (its second) of row lr, which is one operand of
// v_mfma_i32_16x16x64_i8: which 64 of the block's 128 values an instruction
// takes is free, as A and B agree.  B goes first, so that a lane owns one
// output row and four consecutive columns of a sub-tile.
//
// A block takes two phases of TM TN products each.  The first multiplies the
// first halves, while the second halves' fragments are read; it ends with the
// block's only barrier, behind which its stage is free and the next block's has
// landed.  The second multiplies those, while the next block's first halves are
// read and the block S ahead is loaded.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int S_, int GROUP_M_>
struct Int8Tile {
    static constexpr int BM = BM_, BN = BN_, S = S_;
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, kWaves = WAVES_M * WAVES_N;
    static constexpr int kThreads = 64 * kWaves, kGroupM = GROUP_M_;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;  // of a wave
    static constexpr int kStage = (BM + BN) * 128;
    static constexpr int kLoadsA = BM / 8 / kWaves, kLoadsB = (BN / 8 + kWaves - 1) / kWaves;
    static constexpr int kLoads = kLoadsA + kLoadsB;  // of a K block; some waves have one less where kUneven
    static constexpr bool kUneven = BN / 8 % kWaves != 0;
    // the bf16 output tile on its way out: row pitch in 16-byte chunks
    static constexpr int kPitchChunks = BN <= 128 ? 16 : 32;
    static constexpr int kSmem = S * kStage > BM * kPitchChunks * 16 ? S * kStage : BM * kPitchChunks * 16;
    static_assert(WM % 16 == 0 && WN % 16 == 0 && BN <= 256, "whole sub-tiles, output pitch");
    static_assert(BM % (8 * kWaves) == 0 && BN % 8 == 0 && (!kUneven || S == 2), "waits count every wave's loads");
    static_assert(kSmem <= 160 * 1024 && kLoads * (S - 1) < 64, "LDS, vmcnt range");
};

template <class T, bool kGrouped>
__global__ __launch_bounds__(T::kThreads, T::kWaves / 4) void int8_gemm_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ sa, const uint8_t* __restrict__ B,
    const float* __restrict__ sb, uint16_t* __restrict__ D, const int32_t* __restrict__ layout, int64_t rows, int64_t N,
    int64_t K, int64_t G, int m_blocks, int n_blocks) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int KB = (int)(K >> 7);
    const int lr = lane & 15, lg = lane >> 4;
    const int wrow = wave / T::WAVES_N * T::WM, wcol = wave % T::WAVES_N * T::WN;
    const int sub = lane >> 3, lchunk = (lane & 7) ^ sub;
    const uint32_t offRow = (uint32_t)(wave * 8 + sub) * (uint32_t)K + lchunk * 16;
    const int chunk_lo = (lg ^ (lr & 7)) << 4, chunk_hi = chunk_lo ^ 64;
    const int fragA = (wrow + lr) * 128, fragB = T::BM * 128 + (wcol + lr) * 128;

    TileInfo ti;
    ti.ok0 = ti.ok1 = 0;
    ti.g = 0;
    auto compute = [&]() __attribute__((always_inline)) {
        const int vn = (int)min<int64_t>(T::BN, N - ti.n0);
        const uint8_t* tileA = A + ti.arow0 * K;
        const uint8_t* tileB = B + ((int64_t)ti.g * N + ti.n0) * K;
        // a wave's load q of block kb: rows [8 (wave + kWaves q), +8) of A, then of B;
        // blocks past the last one get an empty buffer, and so count like the others
        auto issue = [&](int kb, int st, int q0, int q1) __attribute__((always_inline)) {
            const v4u ra = buffer_rsrc(tileA + kb * 128, kb < KB ? (uint32_t)ti.valid * (uint32_t)K - kb * 128 : 0u);
            const v4u rb = buffer_rsrc(tileB + kb * 128, kb < KB ? (uint32_t)vn * (uint32_t)K - kb * 128 : 0u);
            uint8_t* const to = smem + st * T::kStage + wave * 1024;
            constexpr int kRows = 8 * T::kWaves;  // of a load of every wave
#pragma unroll
            for (int q = q0; q < q1; ++q) {
                if (q < T::kLoadsA)
                    load_lds_16(ra, offRow + (uint32_t)(q * kRows) * (uint32_t)K, to + q * kRows * 128);
                else if (!T::kUneven || wave + (q - T::kLoadsA) * T::kWaves < T::BN / 8)
                    load_lds_16(rb, offRow + (uint32_t)((q - T::kLoadsA) * kRows) * (uint32_t)K, to + q * kRows * 128);
            }
        };
        v4i acc[T::TM][T::TN];
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
#pragma unroll
            for (int j = 0; j < T::TN; ++j) acc[i][j] = v4i{0, 0, 0, 0};
        v4i a[2][T::TM], b[2][T::TN];
        auto read_b = [&](const uint8_t* st, int chunk, int set, int j) __attribute__((always_inline)) {
            b[set][j] = *reinterpret_cast<const v4i*>(st + fragB + j * 2048 + chunk);
        };
        auto read_a = [&](const uint8_t* st, int chunk, int set, int i) __attribute__((always_inline)) {
            a[set][i] = *reinterpret_cast<const v4i*>(st + fragA + i * 2048 + chunk);
        };
        // the products of one set, a row of sub-tiles at a time, with the next
        // set's reads (and, kLoad, the loads of a block) between them
        auto phase = [&](auto which, const uint8_t* next, int chunk, auto load, int kb, int st) __attribute__((always_inline)) {
            constexpr int set = decltype(which)::value;
            constexpr bool kLoad = decltype(load)::value;
            constexpr int kRead = (T::TN + T::TM + T::TM - 1) / T::TM;  // reads a row
            constexpr int kEach = (T::kLoads + T::TM - 1) / T::TM;
#pragma unroll
            for (int i = 0; i < T::TM; ++i) {
#pragma unroll
                for (int r = i * kRead; r < (i + 1) * kRead; ++r) {
                    if (r < T::TN)
                        read_b(next, chunk, set ^ 1, r);
                    else if (r < T::TN + T::TM)
                        read_a(next, chunk, set ^ 1, r - T::TN);
                }
                if constexpr (kLoad) issue(kb, st, i * kEach, min((i + 1) * kEach, T::kLoads));
#pragma unroll
                for (int j = 0; j < T::TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[set][j], a[set][i], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        using std::integral_constant;
        using First = integral_constant<int, 0>;
        using Second = integral_constant<int, 1>;

#pragma unroll
        for (int s = 0; s < T::S; ++s) issue(s, s, 0, T::kLoads);
        wait_vmcnt<T::kUneven ? 0 : T::kLoads*(T::S - 1)>();
        lds_barrier();
#pragma unroll
        for (int j = 0; j < T::TN; ++j) read_b(smem, chunk_lo, 0, j);
#pragma unroll
        for (int i = 0; i < T::TM; ++i) read_a(smem, chunk_lo, 0, i);
        int st = 0;
        for (int kb = 0; kb < KB; ++kb) {
            const int nx = st + 1 == T::S ? 0 : st + 1;
            phase(First{}, smem + st * T::kStage, chunk_hi, std::false_type{}, 0, 0);
            wait_vmcnt_lgkm0<T::kLoads*(T::S - 2)>();  // the stage has been read, the next block's has landed
            lds_barrier();
            phase(Second{}, smem + nx * T::kStage, chunk_lo, std::true_type{}, kb + T::S, st);
            st = nx;
        }
        wait_vmcnt_lgkm0<0>();  // the empty loads of the last blocks have retired
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
            const int row = wrow + 16 * i + lr;
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
    };

    if constexpr (!kGrouped) {
        const int tile = xcd_tile(blockIdx.x, m_blocks * n_blocks);
        if (tile < 0) return;
        const int span = T::kGroupM * n_blocks;
        const int first_m = (tile / span) * T::kGroupM;
        const int gm = min(m_blocks - first_m, T::kGroupM);
        const int in_span = tile % span;
        ti.m0 = (first_m + in_span % gm) * T::BM;
        ti.n0 = (in_span / gm) * T::BN;
        ti.arow0 = ti.m0;
        ti.valid = (int)min<int64_t>(T::BM, rows - ti.m0);
        compute();
    } else {
        // A buffer of the most rows that any choice of experts needs is mostly
        // padding behind the last expert's: a workgroup walks the tiles (the
        // columns of a block first), looking at as many blocks at once as it has waves.
        static_assert(T::BM == 128, "one group per 128-row block");
        int* const ahead = reinterpret_cast<int*>(smem + T::kSmem);
        const int64_t tiles = (int64_t)m_blocks * n_blocks;
        for (int64_t t0 = blockIdx.x; t0 < tiles; t0 += T::kWaves * (int64_t)gridDim.x) {
            const int64_t mine = t0 + wave * (int64_t)gridDim.x;
            int any = 0;
            if (mine < tiles) {
                const int32_t* const ids = layout + mine / n_blocks * 128;
                const int id0 = ids[lane], id1 = ids[64 + lane];
                any = __ballot((id0 >= 0 && id0 < G) || (id1 >= 0 && id1 < G)) != 0;
            }
            if (lane == 0) ahead[wave] = any;
            __syncthreads();
            int todo = 0;
#pragma unroll
            for (int w = 0; w < T::kWaves; ++w) todo |= ahead[w] << w;
            todo = __builtin_amdgcn_readfirstlane(todo);
            __syncthreads();
            while (todo != 0) {
                const int w = __builtin_ctz(todo);
                todo &= todo - 1;
                const int64_t t = t0 + w * (int64_t)gridDim.x;
                ti.m0 = (int)(t / n_blocks) * T::BM;
                ti.n0 = (int)(t % n_blocks) * T::BN;
                ti.arow0 = ti.m0;
                ti.valid = T::BM;
                // once per id among the block's rows, the largest first
                int below = (int)min<int64_t>(G, 0x7fffffff);
                while (block_group(layout, G, below, lane, ti)) {
                    compute();
                    below = ti.g;
                    __syncthreads();  // the staged tile has been stored before the next loads
                }
            }
        }
    }
}

template <class T, bool kGrouped>
static dg_status launch_tiled(const Int8Args& a, hipStream_t stream) {
    const int64_t m_blocks = (a.rows + T::BM - 1) / T::BM, n_blocks = (a.N + T::BN - 1) / T::BN;
    int64_t grid = (m_blocks * n_blocks + kNumXcds - 1) / kNumXcds * kNumXcds;
    if (kGrouped) grid = std::min<int64_t>(grid, device_cus());
    if (!grid_fits(grid, T::kThreads)) return DG_ERR_SHAPE;
    // per-lane 32-bit offsets into a tile's rows of K bytes: K < 2^17
    hipLaunchKernelGGL((int8_gemm_kernel<T, kGrouped>), dim3((unsigned)grid), dim3(T::kThreads), T::kSmem + 64, stream,
                       reinterpret_cast<const uint8_t*>(a.A), a.sa, reinterpret_cast<const uint8_t*>(a.B), a.sb, a.D,
                       a.layout, a.rows, a.N, a.K, a.G, (int)m_blocks, (int)n_blocks);
    return launched();
}

// The product of up to 16 rows: bound by the weights, or by a load's latency.
// A workgroup takes 16 CN columns and all rows, its waves every eighth K block
// each, straight from memory into fragments (a lane's two operands of a block
// are 32 bytes of its row, so that a wave reads whole lines), without a barrier
// before the shares of the sums, which are exact in any order, are added in LDS.
// 1 x 7168 x 2048: 5.7 us, 5.9 in the narrowest tiles, of which a launch alone
// takes 2.5 and 15 MB at a copy's rate 3; 1 x 2112 x 7168, where those tiles are
// few and their K blocks follow each other: 6.4 against 11.4.  With 32 rows, two
// fragments of A for one of B, it gained nothing (11.9 against 11.6).
template <int CN>
__global__ __launch_bounds__(512) void int8_few_rows_kernel(const uint8_t* __restrict__ A, const float* __restrict__ sa,
                                                            const uint8_t* __restrict__ B, const float* __restrict__ sb,
                                                            uint16_t* __restrict__ D, int M, int64_t N, int64_t K) {
    constexpr int W = 8, U = 2;  // waves; K blocks whose loads a wave issues together
    __shared__ v4i part[W][CN][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int KB = (int)(K >> 7);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * CN);
    // rows and columns past the last one read the last one again; their sums go nowhere
    const uint8_t *const pa = A + (int64_t)min(lr, M - 1) * K + 32 * lg, *pb[CN];
#pragma unroll
    for (int c = 0; c < CN; ++c) pb[c] = B + min<int64_t>(n0 + 16 * c + lr, N - 1) * K + 32 * lg;
    // the wave that adds up column tile c: row lr, columns 4 lg .. +3 of it
    const int64_t n = n0 + 16 * wave + 4 * lg;
    const bool adds = wave < CN && lr < M && n < N;
    const float row_scale = adds ? sa[lr] : 0.0f;
    const v4f col_scale = adds ? *reinterpret_cast<const v4f*>(sb + n) : v4f{0.f, 0.f, 0.f, 0.f};
    v4i acc[CN];
#pragma unroll
    for (int c = 0; c < CN; ++c) acc[c] = v4i{0, 0, 0, 0};
    for (int kb0 = wave; kb0 < KB; kb0 += W * U) {
        v4i a[U][2], b[U][CN][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * W;
            if (kb >= KB) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int c = 0; c < CN; ++c) b[u][c][h] = *reinterpret_cast<const v4i*>(pb[c] + kb * 128 + 16 * h);
                a[u][h] = *reinterpret_cast<const v4i*>(pa + kb * 128 + 16 * h);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kb0 + u * W >= KB) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < CN; ++c)
                    acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[u][c][h], a[u][h], acc[c], 0, 0, 0);
        }
    }
#pragma unroll
    for (int c = 0; c < CN; ++c) part[wave][c][lane] = acc[c];
    __syncthreads();
    if (!adds) return;
    v4i sum = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < W; ++w) sum += part[w][wave][lane];
    v2u packed;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const v2f v = {(row_scale * col_scale[2 * h]) * (float)sum[2 * h],
                       (row_scale * col_scale[2 * h + 1]) * (float)sum[2 * h + 1]};
        packed[h] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf));
    }
    *reinterpret_cast<v2u*>(D + (int64_t)lr * N + n) = packed;
}

template <int CN>
static dg_status launch_few_rows(const Int8Args& a, hipStream_t stream) {
    const int64_t grid = (a.N + 16 * CN - 1) / (16 * CN);
    if (!grid_fits(grid, 512)) return DG_ERR_SHAPE;
    hipLaunchKernelGGL((int8_few_rows_kernel<CN>), dim3((unsigned)grid), dim3(512), 0, stream,
                       reinterpret_cast<const uint8_t*>(a.A), a.sa, reinterpret_cast<const uint8_t*>(a.B), a.sb, a.D,
                       (int)a.rows, a.N, a.K);
    return launched();
}

using Int8Large = Int8Tile<256, 256, 2, 4, 2, 4>;
using Int8Wide192 = Int8Tile<256, 192, 4, 2, 2, 4>;
using Int8Wide160 = Int8Tile<256, 160, 4, 2, 2, 4>;
using Int8Rows128 = Int8Tile<128, 256, 2, 4, 3, 8>;
using Int8Square128 = Int8Tile<128, 128, 2, 4, 4, 8>;
using Int8Tall64 = Int8Tile<128, 64, 2, 2, 4, 8>;
using Int8Square64 = Int8Tile<64, 64, 2, 2, 4, 8>;
using Int8Narrow = Int8Tile<64, 32, 2, 2, 4, 8>;

dg_status launch_int8_gemm(const Int8Args& a, hipStream_t stream) {
    if (a.layout != nullptr) return launch_tiled<Int8Rows128, true>(a, stream);
    const int64_t cus = device_cus();
    // 32 columns a workgroup where they are enough for the CUs (1 x 7168 x 2048:
    // 5.7 us, 6.3 with 16), else 16 (8 x 4096 x 7168: 7.8, 10.7 with 32)
    if (a.rows <= 16) return a.N / 32 * 8 >= cus * 7 ? launch_few_rows<2>(a, stream) : launch_few_rows<1>(a, stream);
    // The tile shape with the least estimated time: rounds of one tile a CU
    // times what a K block of the shape takes, in ns, from whole launches of
    // one round (K 2048 and 7168, from 64 x 7168 to 4096 x 2112 columns) and of
    // several (4096 x 7168 x 2048, 8192^3).
    struct Shape { int bm, bn, ns; };
    static const Shape kShapes[] = {{256, 256, 1580}, {256, 192, 1250}, {256, 160, 1070}, {128, 256, 890},
                                    {128, 128, 530},  {128, 64, 320},   {64, 64, 200},    {64, 32, 155}};
    int best = 0;
    int64_t least = INT64_MAX;
    for (int i = 0; i < 8; ++i) {
        const Shape& sh = kShapes[i];
        const int64_t tiles = ((a.rows + sh.bm - 1) / sh.bm) * ((a.N + sh.bn - 1) / sh.bn);
        const int64_t cost = (tiles + cus - 1) / cus * sh.ns;
        if (cost < least) {
            least = cost;
            best = i;
        }
    }
    switch (best) {
        case 0: return launch_tiled<Int8Large, false>(a, stream);
        case 1: return launch_tiled<Int8Wide192, false>(a, stream);
        case 2: return launch_tiled<Int8Wide160, false>(a, stream);
        case 3: return launch_tiled<Int8Rows128, false>(a, stream);
        case 4: return launch_tiled<Int8Square128, false>(a, stream);
        case 5: return launch_tiled<Int8Tall64, false>(a, stream);
        case 6: return launch_tiled<Int8Square64, false>(a, stream);
        default: return launch_tiled<Int8Narrow, false>(a, stream);
    }
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
