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

// A tile.  A K block is 128 bytes a row, loaded straight from memory into one
// of S stages of LDS, 16-byte chunk c of row r at c ^ (r & 7).  Lane (lr, lg) of
// a fragment read takes chunk lg (the block's first half) or lg + 4 (its second)
// of row lr, which is one operand of v_mfma_i32_16x16x64_i8: which 64 of the
// block's 128 values an instruction takes is free, as A and B agree.  B goes
// first, so that a lane owns one output row and four consecutive columns of a
// sub-tile.
//
// A block takes two phases of TM TN products each.  The first multiplies the
// first halves, while the second halves' fragments are read; it ends with the
// block's only barrier, behind which its stage is free and the next block's has
// landed.  The second multiplies those, while the next block's first halves are
// read and the block S ahead is loaded.
//
// 256 x 256 in 8 waves: 1.38 us a K block where the products alone (no loads, no
// reads) take 1.05, and 11 us for a tile's beginning, its end and the launch, of
// which the stores of one round of tiles, 34 MB, are 5.  4096 x 7168 x 2048:
// 57 us, 2110 TOPS; 8192^3: 418 us, 2630 (the library's int8 product side by
// side: 69 and 452; on another card 55 and 374 us here, 2940 TOPS).  Tried,
// beside 55: the FP8 kernel's two barriers a block (59.7 us); four waves of 128 x
// 128 with 512 registers each, whose sums the compiler moves about (78); 32 x 32
// x 32 products (64); the loads at the second phase's beginning instead of spread
// over it (59-60); a barrier in the middle of the first phase for earlier loads
// (62).
//
// Where few tiles leave CUs without one, a K block's latency bounds a tile, and
// PARTS groups of waves with stages of their own take every PARTS-th block each;
// their sums, exact in any order, are added in LDS at the end.  64 x 512 x 7168:
// 7.8 us in 32 x 32 by two groups of two waves (8.2 by four; a group of four
// waves alone: 11.4 in 64 x 32, two 10.2).
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int S_, int GROUP_M_, int PARTS_ = 1>
struct Int8Tile {
    static constexpr int BM = BM_, BN = BN_, S = S_;
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, kWaves = WAVES_M * WAVES_N;
    static constexpr int kThreads = 64 * kWaves, kGroupM = GROUP_M_;  // of a group
    static constexpr int kParts = PARTS_, kAllThreads = kThreads * kParts;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;  // of a wave
    static constexpr int kStage = (BM + BN) * 128;
    static constexpr int kLoadsA = BM / 8 / kWaves, kLoadsB = (BN / 8 + kWaves - 1) / kWaves;
    static constexpr int kLoads = kLoadsA + kLoadsB;  // of a K block; some waves have one less where kUneven
    static constexpr bool kUneven = BN / 8 % kWaves != 0;
    // the bf16 output tile on its way out: row pitch in 16-byte chunks
    static constexpr int kPitchChunks = BN <= 128 ? 16 : 32;
    static constexpr int kOut = BM * kPitchChunks * 16;
    static constexpr int kSums = (kParts - 1) * kThreads * TM * TN * 16;  // of the other groups, behind it
    static constexpr int kStages = kParts * S * kStage;
    static constexpr int kSmem = kStages > kOut + kSums ? kStages : kOut + kSums;
    static_assert(WM % 16 == 0 && WN % 16 == 0 && BN <= 256, "whole sub-tiles, output pitch");
    static_assert(BM % (8 * kWaves) == 0 && BN % 8 == 0 && (!kUneven || S == 2), "waits count every wave's loads");
    static_assert(kSmem <= 160 * 1024 && kLoads * (S - 1) < 64, "LDS, vmcnt range");
};

struct Int8Operands {
    const uint8_t* A;
    const float* sa;
    const uint8_t* B;
    const float* sb;
    uint16_t* D;
    int64_t N, K;
};

// The tile at ti, all threads of the workgroup; kRouted: only the rows of ti's
// masks are stored.  LDS is free again when every wave has come back.
template <class T, bool kRouted>
__device__ __forceinline__ void int8_tile(const Int8Operands& p, const TileInfo& ti, uint8_t* smem, int tid) {
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % T::kWaves;
    const int part = T::kParts > 1 ? __builtin_amdgcn_readfirstlane(tid >> 6) / T::kWaves : 0;
    uint8_t* const own = smem + part * (T::S * T::kStage);
    const int lane = tid & 63;
    const uint32_t K = (uint32_t)p.K;  // below 2^17: a tile's rows are addressed with 32-bit offsets
    const int KB = (int)(K >> 7);
    const int lr = lane & 15, lg = lane >> 4;
    const int wrow = wave / T::WAVES_N * T::WM, wcol = wave % T::WAVES_N * T::WN;
    const int sub = lane >> 3, lchunk = (lane & 7) ^ sub;
    const uint32_t offRow = (uint32_t)(wave * 8 + sub) * K + lchunk * 16;
    const int chunk_lo = (lg ^ (lr & 7)) << 4, chunk_hi = chunk_lo ^ 64;
    const int fragA = (wrow + lr) * 128, fragB = T::BM * 128 + (wcol + lr) * 128;
    const int vn = (int)min<int64_t>(T::BN, p.N - ti.n0);
    const uint8_t* const tileA = p.A + ti.arow0 * p.K;
    const uint8_t* const tileB = p.B + ((int64_t)ti.g * p.N + ti.n0) * p.K;
    // a wave's loads [q0, q1) of its group's block i: rows [8 (wave + kWaves q), +8) of A,
    // then of B; blocks past the last one get an empty buffer, and so count like
    // the others
    auto issue = [&](int i, int st, int q0, int q1) __attribute__((always_inline)) {
        const int kb = i * T::kParts + part;
        const v4u ra = buffer_rsrc(tileA + kb * 128, kb < KB ? (uint32_t)ti.valid * K - kb * 128 : 0u);
        const v4u rb = buffer_rsrc(tileB + kb * 128, kb < KB ? (uint32_t)vn * K - kb * 128 : 0u);
        uint8_t* const to = own + st * T::kStage + wave * 1024;
        constexpr int kRows = 8 * T::kWaves;  // of a load of every wave
#pragma unroll
        for (int q = q0; q < q1; ++q) {
            if (q < T::kLoadsA)
                load_lds_16(ra, offRow + (uint32_t)(q * kRows) * K, to + q * kRows * 128);
            else if (!T::kUneven || wave + (q - T::kLoadsA) * T::kWaves < T::BN / 8)
                load_lds_16(rb, offRow + (uint32_t)((q - T::kLoadsA) * kRows) * K, to + q * kRows * 128);
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
    auto phase = [&](auto which, const uint8_t* next, int chunk, auto load, int block, int st) __attribute__((always_inline)) {
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
            if constexpr (kLoad) issue(block, st, min(i * kEach, T::kLoads), min((i + 1) * kEach, T::kLoads));
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[set][j], a[set][i], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, 1>;

#pragma unroll
    for (int s = 0; s < T::S; ++s) issue(s, s, 0, T::kLoads);
    wait_vmcnt<T::kUneven ? 0 : T::kLoads*(T::S - 1)>();
    lds_barrier();
#pragma unroll
    for (int j = 0; j < T::TN; ++j) read_b(own, chunk_lo, 0, j);
#pragma unroll
    for (int i = 0; i < T::TM; ++i) read_a(own, chunk_lo, 0, i);
    int st = 0;
    for (int i = 0; i * T::kParts < KB; ++i) {
        const int nx = st + 1 == T::S ? 0 : st + 1;
        phase(First{}, own + st * T::kStage, chunk_hi, std::false_type{}, 0, 0);
        wait_vmcnt_lgkm0<T::kLoads*(T::S - 2)>();  // the stage has been read, the next block's has landed
        lds_barrier();
        phase(Second{}, own + nx * T::kStage, chunk_lo, std::true_type{}, i + T::S, st);
        st = nx;
    }
    wait_vmcnt_lgkm0<0>();  // the empty loads of the last blocks have retired
    lds_barrier();

    if constexpr (T::kParts > 1) {
        v4i* const sums = reinterpret_cast<v4i*>(smem + T::kOut) + wave * 64 * T::TM * T::TN + lane;
        auto at = [&](int p, int i, int j) { return (p - 1) * T::kThreads * T::TM * T::TN + (i * T::TN + j) * 64; };
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
                if (part > 0) sums[at(part, i, j)] = acc[i][j];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
#pragma unroll
                for (int p = 1; p < T::kParts; ++p)
                    if (part == 0) acc[i][j] += sums[at(p, i, j)];
    }

    // epilogue, of the first group: scales by row and column, rounding, and out through LDS
    v4f col_scale[T::TN];
#pragma unroll
    for (int j = 0; j < T::TN; ++j) {
        const int64_t col = min<int64_t>(ti.n0 + wcol + 16 * j + 4 * lg, p.N - 4);
        col_scale[j] = *reinterpret_cast<const v4f*>(p.sb + (int64_t)ti.g * p.N + col);
    }
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
        if (part > 0) continue;
        const int row = wrow + 16 * i + lr;
        const float row_scale = p.sa[ti.arow0 + min(row, ti.valid - 1)];
#pragma unroll
        for (int j = 0; j < T::TN; ++j) {
            v4f v;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = (row_scale * col_scale[j][q]) * (float)acc[i][j][q];
            stage_bf16<T>(smem, row, wcol + 16 * j + 4 * lg, v);
        }
    }
    __syncthreads();
    if (part == 0) store_staged<T, kRouted>(smem, tid, ti, p.D, p.N);
}

// The dense form: tiles of shape T over columns [0, split), of shape U behind
// them, whose workgroups (from `first` on) come last.  Two shapes may leave less
// of the last round idle than one.
template <class T, class U>
__global__ __launch_bounds__(T::kAllThreads, T::kAllThreads / 256) void int8_gemm_kernel(Int8Operands p, int64_t rows,
                                                                                         int64_t split, unsigned first) {
    static_assert(T::kAllThreads == U::kAllThreads, "one workgroup size");
    extern __shared__ __align__(1024) uint8_t smem[];
    auto run = [&](auto shape, int block, int64_t from, int64_t to) __attribute__((always_inline)) {
        using X = decltype(shape);
        const int m_blocks = (int)((rows + X::BM - 1) / X::BM), n_blocks = (int)((to - from + X::BN - 1) / X::BN);
        const int tile = xcd_tile(block, m_blocks * n_blocks);
        if (tile < 0) return;
        TileInfo ti;
        ti.ok0 = ti.ok1 = 0;
        ti.g = 0;
        const int span = X::kGroupM * n_blocks;
        const int first_m = (tile / span) * X::kGroupM;
        const int gm = min(m_blocks - first_m, X::kGroupM);
        const int in_span = tile % span;
        ti.m0 = (first_m + in_span % gm) * X::BM;
        ti.n0 = (int)from + (in_span / gm) * X::BN;
        ti.arow0 = ti.m0;
        ti.valid = (int)min<int64_t>(X::BM, rows - ti.m0);
        int8_tile<X, false>(p, ti, smem, threadIdx.x);
    };
    if constexpr (std::is_same<T, U>::value) {
        run(T{}, blockIdx.x, 0, p.N);
    } else {
        if (blockIdx.x < first)
            run(T{}, blockIdx.x, 0, split);
        else
            run(U{}, blockIdx.x - first, split, p.N);
    }
}

// The contiguous-grouped form.  A buffer of the most rows that any choice of
// experts needs is mostly padding behind the last expert's, so the 128-row
// blocks that hold rows are found first, by every workgroup for itself (in
// windows of kWindow blocks), and their tiles, the columns of a block first,
// are shared out evenly: with one workgroup per tile of the buffer, in order,
// 4096 rows in a buffer of 33664 were left to one of the 8 XCDs (829 us for 8
// experts of 4096 x 7168).  Tiles that are left over behind the whole rounds are
// cut in two (T2) or four (T4) where that takes less than a round of whole ones,
// and blocks of few rows in eight (T8: fewer rows, K in parts).  Rows behind an
// id's last one in a block are not loaded (16 blocks of 8 rows, 1024 x 7168: 24.7
// us, 39.6 with them).
template <class T, class T2, class T4, class T8>
__global__ __launch_bounds__(T::kThreads, T::kWaves / 4) void int8_grouped_kernel(Int8Operands p,
                                                                                  const int32_t* __restrict__ layout,
                                                                                  int64_t rows, int64_t G) {
    static_assert(T::BM == 128 && T2::BM == 128 && T4::BM == 128 && T8::BM < 128, "one group per 128-row block");
    static_assert(T::kSmem >= T2::kSmem && T::kSmem >= T4::kSmem && T::kSmem >= T8::kSmem, "LDS of every shape");
    static_assert(T2::BN * 2 == T::BN && T4::BN * 4 == T::BN && T8::BN * 8 == T::BN, "halves, quarters and eighths");
    static_assert(T::kAllThreads == T2::kAllThreads && T::kAllThreads == T4::kAllThreads &&
                      T::kAllThreads == T8::kAllThreads,
                  "one workgroup size");
    constexpr int kWindow = 4096;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint16_t used[kWindow / 16];  // a bit per block: whether it holds a row
    __shared__ int deep[T::kWaves];                       // of a wave's blocks: whether one holds a row from T8::BM on
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m_blocks = rows / 128;
    const int n_blocks = (int)((p.N + T::BN - 1) / T::BN);
    const int grid = (int)gridDim.x;
    for (int64_t w0 = 0; w0 < m_blocks; w0 += kWindow) {
        const int blocks = (int)min<int64_t>(kWindow, m_blocks - w0), words = (blocks + 63) / 64;
        // a load covers two blocks, 32 lanes of four ids each; eight loads at once,
        // those past the last block of its own ids again
        uint64_t lower = 0;
        for (int b0 = wave * 16; b0 < words * 64; b0 += T::kWaves * 16) {
            int4 id[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int b = min(b0 + 2 * i + (lane >> 5), blocks - 1);
                id[i] = *reinterpret_cast<const int4*>(layout + (w0 + b) * 128 + (lane & 31) * 4);
            }
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                auto valid = [&](int e) { return (uint32_t)e < (uint32_t)G; };
                const uint64_t any = __ballot(valid(id[i].x) || valid(id[i].y) || valid(id[i].z) || valid(id[i].w));
                lower |= any & ~(((uint64_t(1) << (T8::BM / 4)) - 1) * 0x100000001ull);
                bits |= (((uint32_t)any != 0 ? 1u : 0u) | ((any >> 32) != 0 ? 2u : 0u)) << (2 * i);
            }
            bits &= b0 >= blocks ? 0u : blocks - b0 >= 16 ? 0xffffu : (1u << (blocks - b0)) - 1u;
            if (lane == 0) used[b0 / 16] = (uint16_t)bits;
        }
        if (lane == 0) deep[wave] = lower != 0;
        __syncthreads();
        int shallow = 1;
#pragma unroll
        for (int w = 0; w < T::kWaves; ++w) shallow &= deep[w] == 0;
        // lane l holds word l of the window's blocks, and how many are used up to its end
        const uint64_t word = lane < words ? reinterpret_cast<const uint64_t*>(used)[lane] : 0;
        int upto = __popcll(word);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int below = __shfl_up(upto, d, 64);
            if (lane >= d) upto += below;
        }
        const int before = upto - __popcll(word);
        const int64_t tiles = (int64_t)__builtin_amdgcn_readlane(upto, 63) * n_blocks;
        const int left = (int)(tiles % grid);
        // us a K block and round: 0.95 whole, 0.6 halves, 0.43 quarters
        const int cost2 = (2 * left + grid - 1) / grid * 60, cost4 = (4 * left + grid - 1) / grid * 43;
        // eighths of the first 32 rows, if no block has more and they take one
        // round (12 blocks of 512 x 7168: 13.4 us, 20.8 in quarters; more rounds
        // gain nothing)
        const bool eighths = __builtin_amdgcn_readfirstlane(shallow) != 0 && 8 * tiles <= grid;
        const int cut = eighths ? 8 : left == 0 || min(cost2, cost4) >= 95 ? 1 : cost2 <= cost4 ? 2 : 4;
        const int64_t whole = cut > 1 ? tiles - left : tiles;
        auto run = [&](auto shape, int64_t t, int part) __attribute__((always_inline)) {
            using X = decltype(shape);
            // the block: which word holds the k-th used one, then which bit
            const int k = (int)(t / n_blocks);
            const int at = __builtin_ctzll(__ballot(before <= k && k < upto));
            uint64_t bits = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)word, at) |
                            (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(word >> 32), at) << 32;
            for (int skip = k - __builtin_amdgcn_readlane(before, at); skip > 0; --skip) bits &= bits - 1;
            TileInfo ti;
            ti.m0 = (int)(w0 + at * 64 + __builtin_ctzll(bits)) * 128;
            ti.n0 = (int)(t % n_blocks) * T::BN + part * X::BN;
            if (ti.n0 >= p.N) return;
            ti.arow0 = ti.m0;
            // once per id among the block's rows, the largest first
            const int id0 = layout[ti.m0 + lane], id1 = layout[ti.m0 + 64 + lane];
            for (int64_t below = G;;) {
                auto usable = [&](int id) { return id >= 0 && id < below; };
                const int largest = max(usable(id0) ? id0 : -1, usable(id1) ? id1 : -1);
                ti.g = (int)wave_max((uint32_t)(largest + 1)) - 1;
                if (ti.g < 0) break;
                ti.ok0 = __ballot(id0 == ti.g);
                ti.ok1 = __ballot(id1 == ti.g);
                // rows behind the id's last one are not loaded
                ti.valid = ti.ok1 != 0 ? 128 - __builtin_clzll(ti.ok1) : 64 - __builtin_clzll(ti.ok0);
                int8_tile<X, true>(p, ti, smem, tid);
                __syncthreads();  // the staged tile has been stored before the next loads
                below = ti.g;
            }
        };
        for (int64_t t = blockIdx.x; t < whole; t += grid) run(T{}, t, 0);
        if (cut == 2)
            for (int i = blockIdx.x; i < left * 2; i += grid) run(T2{}, whole + i / 2, i % 2);
        else if (cut == 4)
            for (int i = blockIdx.x; i < left * 4; i += grid) run(T4{}, whole + i / 4, i % 4);
        else if (cut == 8)
            for (int i = blockIdx.x; i < left * 8; i += grid) run(T8{}, whole + i / 8, i % 8);
        __syncthreads();  // the bits have been read
    }
}

template <class T, class U>
static dg_status launch_tiled(const Int8Args& a, int64_t split, hipStream_t stream) {
    auto tiles = [&](int64_t bm, int64_t bn, int64_t columns) {
        return ((a.rows + bm - 1) / bm * ((columns + bn - 1) / bn) + kNumXcds - 1) / kNumXcds * kNumXcds;
    };
    const int64_t first = tiles(T::BM, T::BN, split), grid = first + tiles(U::BM, U::BN, a.N - split);
    if (!grid_fits(grid, T::kAllThreads)) return DG_ERR_SHAPE;
    const Int8Operands p{reinterpret_cast<const uint8_t*>(a.A), a.sa, reinterpret_cast<const uint8_t*>(a.B), a.sb, a.D,
                         a.N, a.K};
    hipLaunchKernelGGL((int8_gemm_kernel<T, U>), dim3((unsigned)grid), dim3(T::kAllThreads),
                       T::kSmem > U::kSmem ? T::kSmem : U::kSmem, stream, p, a.rows, split, (unsigned)first);
    return launched();
}

// The product of up to 16 rows: bound by the weights, or by a load's latency.
// A workgroup takes 16 CN columns and all rows, its waves every eighth K block
// each, straight from memory into fragments (a lane's two operands of a block
// are 32 bytes of its row, so that a wave reads whole lines), without a barrier
// before the shares of the sums, which are exact in any order, are added in LDS.
// A call from a graph, in tiles in brackets: 1 x 7168 x 2048 5.2 us (5.8), of
// which the kernel is 4.6, a launch alone 2.5 and 15 MB at a copy's rate 3;
// 1 x 2112 x 7168 6.6 (10.0), 8 x 4096 x 7168 8.2 (10.7); 17 rows take tiles, 6.0.
// With two or four row tiles its loads, 16 bytes of a row a lane, bound it
// (64 x 2112 x 7168: 15 and 22 us).
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
using Int8Parted = Int8Tile<32, 32, 2, 1, 4, 8, 2>;
using Int8Quarter = Int8Tile<128, 64, 4, 2, 4, 8>;   // of Int8Rows128; Int8Square128 is half of it
using Int8Eighth = Int8Tile<32, 32, 2, 1, 4, 8, 4>;  // of its first 32 rows

static dg_status launch_grouped(const Int8Args& a, hipStream_t stream) {
    using T = Int8Rows128;
    const int64_t tiles = a.rows / 128 * ((a.N + T::BN - 1) / T::BN) * 8;
    const Int8Operands p{reinterpret_cast<const uint8_t*>(a.A), a.sa, reinterpret_cast<const uint8_t*>(a.B), a.sb, a.D,
                         a.N, a.K};
    hipLaunchKernelGGL((int8_grouped_kernel<T, Int8Square128, Int8Quarter, Int8Eighth>),
                       dim3((unsigned)std::min<int64_t>(tiles, device_cus())), dim3(T::kThreads), T::kSmem, stream, p,
                       a.layout, a.rows, a.G);
    return launched();
}

dg_status launch_int8_gemm(const Int8Args& a, hipStream_t stream) {
    if (a.layout != nullptr) return launch_grouped(a, stream);
    const int64_t cus = device_cus();
    // 32 columns a workgroup where they are enough for the CUs (16 x 7168 x 2048:
    // 5.7 us, 6.6 with 16), else 16 (8 x 4096 x 7168: 8.2, 11.0 with 32)
    if (a.rows <= 16) return a.N / 32 * 8 >= cus * 7 ? launch_few_rows<2>(a, stream) : launch_few_rows<1>(a, stream);
    // The tile shape with the least estimated time: rounds of one tile a CU
    // times what a K block of the shape takes, in ns, from whole launches of
    // one round (K 2048 and 7168, from 64 x 7168 to 4096 x 2112 columns) and of
    // several (4096 x 7168 x 2048, 8192^3).
    struct Shape { int bm, bn, ns; };
    static const Shape kShapes[] = {{256, 256, 1580}, {256, 192, 1250}, {256, 160, 1070}, {128, 256, 890},
                                    {128, 128, 530},  {128, 64, 320},   {64, 64, 200},    {64, 32, 155},
                                    {32, 32, 88}};
    auto rounds = [&](const Shape& sh, int64_t columns) {
        return ((a.rows + sh.bm - 1) / sh.bm * ((columns + sh.bn - 1) / sh.bn) + cus - 1) / cus;
    };
    int best = 0;
    int64_t least = INT64_MAX, split = a.N;
    // not the last one for short sums, as adding up its parts takes 0.2 us, three
    // K blocks' time, nor in a second round (96 x 5000 x 2048: 7.0 us for 6.7)
    const int shapes = a.K < 640 || rounds(kShapes[8], a.N) > 1 ? 8 : 9;
    for (int i = 0; i < shapes; ++i) {
        const int64_t cost = rounds(kShapes[i], a.N) * kShapes[i].ns;
        if (cost < least) {
            least = cost;
            best = i;
        }
    }
    // or as many rounds of 256 x 256 tiles as are whole, and 192 or 160 columns
    // behind them
    const int64_t whole = rounds(kShapes[0], a.N) - 1, m_blocks = (a.rows + 255) / 256;
    for (int i = 1; i <= 2 && whole > 0 && m_blocks <= whole * cus; ++i) {
        const int64_t at = whole * cus / m_blocks * 256;
        if (at >= a.N) continue;
        const int64_t cost = whole * kShapes[0].ns + rounds(kShapes[i], a.N - at) * kShapes[i].ns;
        if (cost < least) {
            least = cost;
            best = 8 + i;
            split = at;
        }
    }
    switch (best) {
        case 0: return launch_tiled<Int8Large, Int8Large>(a, split, stream);
        case 1: return launch_tiled<Int8Wide192, Int8Wide192>(a, split, stream);
        case 2: return launch_tiled<Int8Wide160, Int8Wide160>(a, split, stream);
        case 3: return launch_tiled<Int8Rows128, Int8Rows128>(a, split, stream);
        case 4: return launch_tiled<Int8Square128, Int8Square128>(a, split, stream);
        case 5: return launch_tiled<Int8Tall64, Int8Tall64>(a, split, stream);
        case 6: return launch_tiled<Int8Square64, Int8Square64>(a, split, stream);
        case 7: return launch_tiled<Int8Narrow, Int8Narrow>(a, split, stream);
        case 8: return launch_tiled<Int8Parted, Int8Parted>(a, split, stream);
        case 9: return launch_tiled<Int8Large, Int8Wide192>(a, split, stream);
        default: return launch_tiled<Int8Large, Int8Wide160>(a, split, stream);
    }
}

// A row by G threads, as the scale needs all of it, with its values held in
// registers up to 8192 columns: bf16 4096 x 7168 23.4 us, 3.8 TB/s (24.0 loaded
// twice), fp32 29.7 us, 4.9 TB/s (43).  A wave each for short rows: 16384 x 1024
// 11.9 us, 16.3 by a workgroup each.
template <bool kBf16, int G, int C>
__global__ __launch_bounds__(256) void quantize_int8_kernel(const void* __restrict__ x, int64_t M, int64_t K,
                                                            uint8_t* __restrict__ q, float* __restrict__ s) {
    __shared__ uint32_t tops[4];
    const int64_t m = blockIdx.x * (int64_t)(256 / G) + threadIdx.x / G;
    if (m >= M) return;  // uniform over the row's threads
    const int id = threadIdx.x % G;
    const float scale = int8_row<G, C>(
        K / 8, id, tops,
        [&](int64_t c, float (&f)[8]) {
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
        },
        [&](int64_t c, const v2u& codes) { *reinterpret_cast<v2u*>(q + m * K + c * 8) = codes; });
    if (id == 0) s[m] = scale;
}

template <bool kBf16>
static dg_status quantize_int8(const void* x, int64_t M, int64_t K, uint8_t* q, float* s, hipStream_t stream) {
    const int64_t grid = K <= 2048 ? (M + 3) / 4 : M;
    if (!grid_fits(grid, 256)) return DG_ERR_SHAPE;
    hipLaunchKernelGGL(K <= 512    ? (quantize_int8_kernel<kBf16, 64, 1>)
                       : K <= 2048 ? (quantize_int8_kernel<kBf16, 64, 4>)
                       : K <= 8192 ? (quantize_int8_kernel<kBf16, 256, 4>)
                                   : (quantize_int8_kernel<kBf16, 256, 0>),
                       dim3((unsigned)grid), dim3(256), 0, stream, x, M, K, q, s);
    return launched();
}

dg_status launch_quantize_int8(const void* x, bool bf16, int64_t M, int64_t K, int8_t* q, float* s, hipStream_t stream) {
    auto* const codes = reinterpret_cast<uint8_t*>(q);
    return bf16 ? quantize_int8<true>(x, M, K, codes, s, stream) : quantize_int8<false>(x, M, K, codes, s, stream);
}

}  // namespace dg
