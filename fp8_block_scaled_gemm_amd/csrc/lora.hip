// A shared projection with each row's own low-rank adapter.  include/dg_ops.h
// has the definition.
//
// Many rows: the adapters' first product (the shrink) here, the second in the
// epilogue of the dense GEMM (gemm.hip).  A few rows: one launch streams the
// shared weights, K split over workgroups, beside the shrink's workgroups; a
// second adds the parts and the adapters' second product.
#include "ops_launch.h"

#include <algorithm>
#include <type_traits>

#include "fewrow.h"

namespace dg {

constexpr int kMaxParts = 4;  // of the shrink's K (8: 14.8 instead of 13.4 us for 64 rows of 64 adapters)

// Shape of the shrink for RT tiles of 16 ranks: RX tiles of 16 rows, W waves
// with a ring of D stages each, a stage being 2 KB per tile of x and of the
// adapter.  Beside the few-row product two workgroups share a CU's LDS; alone,
// a workgroup takes it for itself and reads each adapter for twice the rows.
template <int RT, bool kMany>
struct ShrinkShape {
    static constexpr int RX = kMany && RT <= 4 ? 2 : 1;
    static constexpr int W = kMany ? (RT == 1 ? 8 : 4) : (RT == 8 ? 2 : 4);
    static constexpr int D = kMany ? (RT == 2 ? 4 : RT == 8 ? 2 : 3) : (RT == 1 ? 4 : RT == 2 ? 3 : 2);
    static constexpr int kStage = (RX + RT) * 2048;
    static constexpr int kLds = W * D * kStage;
    static constexpr int kPitch = 16 * RT + 4;
    static_assert(W * 16 * RX * kPitch * 4 <= kLds, "the waves' sums fit the ring");
};

struct ShrinkArgs {
    const uint16_t *x, *lora_a;
    const int32_t* ids;
    float* low;  // [parts][M][R]
    int64_t M, K;
    int L, R;
    int blocks, slots, parts;
    bool grouped;
};

// The rows of block `b` when rows are grouped by adapter: adapters in order,
// each one's rows in order, cut into blocks of kRows.  Every workgroup works
// it out from the ids (a few microseconds, the same in all of them).  Returns
// the adapter, or -1 past the last block; `row` is lane l's row, `n` their
// number.  `lds`: L + kRows + 16 ints, free again on return.
template <int kRows>
__device__ __forceinline__ int find_group(const int32_t* __restrict__ ids, int M, int L, int b, int* lds, int& row,
                                          int& n) {
    int* const count = lds;
    int* const list = lds + L;
    int* const below = list + kRows;  // per wave
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < L; i += threads) count[i] = 0;
    __syncthreads();
    // a thread's ids are consecutive, so ranks follow thread order
    const int per = ((M + threads - 1) / threads + 3) & ~3, r0 = tid * per, r1 = min(r0 + per, M);
    auto each = [&](auto f) __attribute__((always_inline)) {
        for (int r = r0; r < r1; r += 4) {
            int4 v = make_int4(-1, -1, -1, -1);
            if (r + 4 <= M) {
                v = *reinterpret_cast<const int4*>(ids + r);
            } else {
                v.x = ids[r];
                if (r + 1 < M) v.y = ids[r + 1];
                if (r + 2 < M) v.z = ids[r + 2];
            }
            f(r, v.x);
            f(r + 1, v.y);
            f(r + 2, v.z);
            f(r + 3, v.w);
        }
    };
    int same = -1, times = 0;  // runs of one id are counted with one addition
    auto flush = [&]() __attribute__((always_inline)) {
        if (times > 0) atomicAdd(&count[same], times);
    };
    each([&](int, int id) {
        if (id < 0 || id >= L) return;
        if (id == same) {
            ++times;
        } else {
            flush();
            same = id;
            times = 1;
        }
    });
    flush();
    __syncthreads();
    int a = -1, first = 0, total = 0;
    for (int a0 = 0, before = 0; a0 < L; a0 += 64) {
        const int c = a0 + lane < L ? count[a0 + lane] : 0, blocks = (c + kRows - 1) / kRows;
        int upto = blocks;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d, 64);
            if (lane >= d) upto += o;
        }
        const uint64_t past = __ballot(before + upto > b);
        if (past != 0) {
            const int at = __builtin_ctzll(past);
            a = a0 + at;
            total = __builtin_amdgcn_readlane(c, at);
            first = (b - before - __builtin_amdgcn_readlane(upto - blocks, at)) * kRows;
            break;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (a < 0) return -1;
    int mine = 0;
    each([&](int, int id) { mine += id == a; });
    int rank = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(rank, d, 64);
        if (lane >= d) rank += o;
    }
    if (lane == 63) below[wave] = rank;
    __syncthreads();
    rank -= mine;
    for (int w = 0; w < wave; ++w) rank += below[w];
    each([&](int r, int id) {
        if (id == a) {
            if (rank >= first && rank < first + kRows) list[rank - first] = r;
            ++rank;
        }
    });
    __syncthreads();
    n = __builtin_amdgcn_readfirstlane(min(kRows, total - first));
    row = list[min(lane, n - 1)];
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(a);
}

// low[part][m][0..R) = x_m lora_a[a]^T over the part's share of K, for the rows
// m that have an adapter.  A workgroup takes 16 RX rows and one part of K,
// which its waves split; the waves' sums meet in LDS.  With rows grouped by
// adapter they are rows of one adapter.  Without, they are adjacent rows, and
// the workgroup takes the distinct adapters number `slot`, + slots, .. among
// them, one after the other; a product row belongs to one x row only, so rows
// of other adapters are computed beside it and dropped.
//
// 64 columns of bf16 are 128 bytes, so a step of a wave looks like a K block of
// the FP8 products and streams the same way: whole lines straight to a ring of
// the wave's own in LDS (fragment-shaped loads to registers are bound by the
// cache's tag rate, 16 bytes per clock).  4096 rows of K 2048, 8 packed
// prompts, rank 64: 13.1 us; 16.8 MB of x at 1.3 TB/s.  Bound by a workgroup's
// chain of its search for its rows and one pass over K, with 136 workgroups at
// most one to a CU: 120 CUs have none.
template <int RT, bool kMany>
__device__ __forceinline__ void shrink_block(uint8_t* smem, const ShrinkArgs& g, int block, int slot0, int z) {
    using Shape = ShrinkShape<RT, kMany>;
    constexpr int RX = Shape::RX, W = Shape::W, D = Shape::D, kStage = Shape::kStage, kPitch = Shape::kPitch;
    float* const part = reinterpret_cast<float*>(smem);  // [W][16 RX][kPitch], once the ring is done
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4, R = g.R;
    const int64_t m0 = g.grouped ? 0 : (int64_t)block * 16 * RX, K = g.K;
    int rows, id, row = lane;  // lane l: row m0 + row and its adapter
    uint32_t leaders;          // the first row of each distinct adapter
    if (g.grouped) {
        const int a = find_group<16 * RX>(g.ids, (int)g.M, g.L, block, reinterpret_cast<int*>(smem), row, rows);
        if (a < 0) return;
        id = lane < rows ? a : -1;
        leaders = 1;
    } else {
        rows = (int)std::min<int64_t>(16 * RX, g.M - m0);
        id = lane < rows ? g.ids[m0 + lane] : -1;
        if (id < 0 || id >= g.L) id = -1;
        bool first = id >= 0;
#pragma unroll
        for (int d = 0; d < 16 * RX - 1; ++d)
            if (d < lane && __builtin_amdgcn_readlane(id, d) == id) first = false;
        leaders = (uint32_t)__ballot(first);
    }
    const int steps = (int)(K >> 6), shares = g.parts * W, share = z * W + wave;
    const int s0 = (int)((int64_t)share * steps / shares), s1 = (int)((int64_t)(share + 1) * steps / shares);
    // rows past the last one read as zero; K < 2^23, so R <= 128 rows of K bf16
    // fit 31-bit offsets, and grouped rows are below 2^31 bytes of x
    const uint32_t pitch = (uint32_t)K * 2;
    const int reach = __builtin_amdgcn_readfirstlane(g.grouped ? (int)g.M : rows);
    const v4u bufX = buffer_rsrc(g.x + m0 * K, (uint32_t)reach * pitch);
    uint32_t offX[2 * RX];
#pragma unroll
    for (int j = 0; j < 2 * RX; ++j) {
        const int i = 8 * j + (lane >> 3), at = __shfl(row, i, 64);
        offX[j] = i < rows ? (uint32_t)at * pitch + panel_chunk(lane) : kNoRow;
    }
    const uint32_t off = (uint32_t)(lane >> 3) * pitch + panel_chunk(lane);
    uint8_t* const ring = smem + wave * D * kStage;
    const int lo = (lg ^ (lr & 7)) << 4, hi = lo ^ 64;
    for (int n = 0; leaders != 0; ++n, leaders &= leaders - 1) {
        if (n % g.slots != slot0) continue;
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(leaders));
        if (wave < W) {
            const v4u bufA = buffer_rsrc(g.lora_a + (int64_t)a * R * K, (uint32_t)R * pitch);
            auto issue = [&](int s, int slot) __attribute__((always_inline)) {
                uint8_t* const to = ring + slot * kStage;
#pragma unroll
                for (int j = 0; j < 2 * RX; ++j)
                    load_lds_16(bufX, s < s1 ? offX[j] + s * 128 : kNoRow, to + j * 1024);
#pragma unroll
                for (int j = 0; j < 2 * RT; ++j)
                    load_lds_16(bufA, s < s1 ? off + (uint32_t)(8 * j) * pitch + s * 128 : kNoRow,
                                to + RX * 2048 + j * 1024);
            };
            v4f acc[RX][RT];
            clear(acc);
#pragma unroll
            for (int d = 0; d < D - 1; ++d) issue(s0 + d, d);
            int slot = 0;
            for (int s = s0; s < s1; ++s) {
                wait_vmcnt_lgkm0<2 * (RX + RT) * (D - 2)>();
                asm volatile("" ::: "memory");
                issue(s + D - 1, slot == 0 ? D - 1 : slot - 1);
                const uint8_t* const p = ring + slot * kStage + lr * 128;
                v8bf xf[RX][2];
#pragma unroll
                for (int t = 0; t < RX; ++t) {
                    xf[t][0] = *reinterpret_cast<const v8bf*>(p + t * 2048 + lo);
                    xf[t][1] = *reinterpret_cast<const v8bf*>(p + t * 2048 + hi);
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint8_t* const q = p + 2048 * (RX + r);
                    const v8bf a0 = *reinterpret_cast<const v8bf*>(q + lo), a1 = *reinterpret_cast<const v8bf*>(q + hi);
#pragma unroll
                    for (int t = 0; t < RX; ++t) {
                        acc[t][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, xf[t][0], acc[t][r], 0, 0, 0);
                        acc[t][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, xf[t][1], acc[t][r], 0, 0, 0);
                    }
                }
                slot = slot == D - 1 ? 0 : slot + 1;
            }
            wait_vmcnt_lgkm0<0>();
            __syncthreads();
#pragma unroll
            for (int t = 0; t < RX; ++t)
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    *reinterpret_cast<v4f*>(part + ((wave * RX + t) * 16 + lr) * kPitch + 16 * r + 4 * lg) = acc[t][r];
        } else {
            __syncthreads();
        }
        __syncthreads();
        // four ranks a thread
        constexpr int kQuads = 4 * RT;
        for (int i = threadIdx.x; i < 16 * RX * kQuads; i += blockDim.x) {
            const int mi = i / kQuads, r = i % kQuads * 4;
            v4f sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < W; ++w) sum += *reinterpret_cast<const v4f*>(part + (w * 16 * RX + mi) * kPitch + r);
            const int at = __shfl(row, mi, 64);
            if (__shfl(id, mi, 64) == a && r < R)  // R is a multiple of 8
                *reinterpret_cast<v4f*>(g.low + ((int64_t)z * g.M + m0 + at) * R + r) = sum;
        }
        __syncthreads();  // the sums have been read: the ring is free again
    }
}

template <int RT>
__global__ __launch_bounds__((64 * ShrinkShape<RT, true>::W)) void lora_shrink_kernel(ShrinkArgs g) {
    extern __shared__ __align__(1024) uint8_t smem[];
    shrink_block<RT, true>(smem, g, blockIdx.x, blockIdx.y, blockIdx.z);
}

// A few rows: the first workgroups multiply 16 T rows by 128 columns over one
// share of K and leave fp32 parts; the others are the shrink's (in the other
// order 64 rows of 64 adapters take 17.9 us instead of 15.0).  One burst of
// loads has about 2 us of latency, so what counts is that all of B is asked
// for at once: K is split until every CU has a workgroup.  64 rows of
// 2112 x 7168, 64 adapters of rank 32: 13 us for 47 MB, and 5.4 us for the
// combine (15.6 MB); the two products alone would take a copy's rate 11 us.
constexpr int kFewRing = 3;

struct FewArgs {
    const uint8_t* A;
    const void* sa;
    const uint8_t* B;
    const void* sb;
    float* sums;  // [shares][M][N]
    int M, N, K;
    int row_tiles, col_tiles, shares, per;  // per: K blocks of a share, a multiple of 4
};

template <int T, int RT, bool kE8>
__global__ __launch_bounds__(64 * kPanelWaves) void lora_few_kernel(FewArgs f, ShrinkArgs g) {
    using S = typename std::conditional<kE8, uint8_t, float>::type;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int base = f.row_tiles * f.col_tiles * f.shares;
    int b = blockIdx.x;
    if (b >= base) {
        b -= base;
        shrink_block<RT, false>(smem, g, b / (g.slots * g.parts), b / g.parts % g.slots, b % g.parts);
        return;
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4, sub = lane >> 3;
    const int m0 = b % f.row_tiles * 16 * T, n0 = b / f.row_tiles % f.col_tiles * 128;
    const int share = b / (f.row_tiles * f.col_tiles), kb0 = share * f.per;
    const int KB = f.K >> 7, SP = scale_pitch<kE8>(KB), rows = min(16 * T, f.M - m0), cols = min(128, f.N - n0);
    const uint32_t K = (uint32_t)f.K, chunk = panel_chunk(lane), kSz = sizeof(S);
    PanelLoads<1> p;
    // rows and columns past the last ones read as zero
    p.bufA = buffer_rsrc(f.A + (int64_t)m0 * K + kb0 * 128, rows * K - kb0 * 128);
    p.bufB = buffer_rsrc(f.B + (int64_t)n0 * K + kb0 * 128, cols * K - kb0 * 128);
    p.bufS = wave == 0 ? buffer_rsrc(static_cast<const S*>(f.sa) + (int64_t)m0 * SP + kb0, (rows * SP - kb0) * kSz)
                       : buffer_rsrc(static_cast<const S*>(f.sb) + (int64_t)(n0 >> 7) * SP + kb0, (SP - kb0) * kSz);
#pragma unroll
    for (int j = 0; j < 2; ++j) p.offB[j] = (uint32_t)(16 * wave + 8 * j + sub) * K + chunk;
    p.offA[0] = (uint32_t)(8 * wave + sub) * K + chunk;
    p.offS = wave == 0 && lane < rows ? (uint32_t)lane * SP * kSz : wave == 1 && lane == 0 ? 0u : kNoRow;
    v4f acc[T][1];
    panel_product<T, 1, kFewRing, kE8, false>(smem, p, min(f.per, KB - kb0), rows, wave, lane, acc);
    const int col = 16 * wave + 4 * lg;
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (16 * t + lr < rows && col < cols)  // N is a multiple of 8
            *reinterpret_cast<v4f*>(f.sums + ((int64_t)share * f.M + m0 + 16 * t + lr) * f.N + n0 + col) = acc[t][0];
}

// D[m][n] = bf16(sum of the shares + scaling[id] * low_m . lora_b[id][n]): one
// output a thread, 256 columns of one row a workgroup.
template <int RC>  // RC >= R / 8
__global__ __launch_bounds__(256) void lora_combine_kernel(
    const float* __restrict__ sums, const float* __restrict__ low, const uint16_t* __restrict__ lora_b,
    const float* __restrict__ scaling, const int32_t* __restrict__ ids, uint16_t* __restrict__ D, int M, int N,
    int L, int R, int parts, int shares) {
    __shared__ float vec[8 * RC];
    const int m = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x, at = min(n, N - 1);
    const int id = ids[m];
    const bool adapted = id >= 0 && id < L;  // uniform
    float sum = 0;
    v4u b[RC];
    if (adapted) {
        const uint16_t* const pb = lora_b + ((int64_t)id * N + at) * R;
#pragma unroll
        for (int c = 0; c < RC; ++c) b[c] = *reinterpret_cast<const v4u*>(pb + min(8 * c, R - 8));
        if (threadIdx.x < 8 * RC) {
            float v[kMaxParts], s = 0;
#pragma unroll
            for (int p = 0; p < kMaxParts; ++p)
                v[p] = low[((int64_t)min(p, parts - 1) * M + m) * R + min((int)threadIdx.x, R - 1)];
#pragma unroll
            for (int p = 0; p < kMaxParts; ++p) s += p < parts ? v[p] : 0.0f;
            vec[threadIdx.x] = scaling[id] * s;
        }
    }
    const float* const from = sums + (int64_t)m * N + at;
    const int64_t next = (int64_t)M * N;
    int s = 0;
    for (; s + 4 <= shares; s += 4) {
        const float v0 = from[s * next], v1 = from[(s + 1) * next], v2 = from[(s + 2) * next], v3 = from[(s + 3) * next];
        sum += (v0 + v1) + (v2 + v3);
    }
    for (; s < shares; ++s) sum += from[s * next];
    if (adapted) {
        __syncthreads();
        float term = 0;
#pragma unroll
        for (int c = 0; c < RC; ++c) {
            if (8 * c >= R) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                term = fmaf(vec[8 * c + 2 * q], __uint_as_float(b[c][q] << 16), term);
                term = fmaf(vec[8 * c + 2 * q + 1], __uint_as_float(b[c][q] & 0xffff0000u), term);
            }
        }
        sum += term;
    }
    // N is a multiple of 8: the even lane of a pair stores both columns
    const v2f pair = {sum, __shfl_xor(sum, 1, 64)};
    if ((n & 1) == 0 && n < N)
        *reinterpret_cast<uint32_t*>(D + (int64_t)m * N + n) =
            __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, v2bf));
}

// What a call launches, from its sizes; M >= 1 (no rows: no launch, no plan).
struct LoraPlan {
    bool few;
    int T, row_tiles, col_tiles, shares, per;  // few rows
    int64_t blocks;                            // the shrink
    int slots, parts;
    bool grouped;
    int64_t low, sums, total;                  // workspace, in bytes from its start
    LoraPlan(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
        // The few-row form splits K over workgroups and reads each row's adapter
        // by itself: its second launch costs about M N R.  The dense tiles walk K
        // whole and take a step for each adapter among a tile's rows, at most L.
        // So M N R / K decides, against a limit that grows with L.  Measured, few
        // rows / dense tiles, us: 300 x 2048 x 1024, rank 64, 12 adapters in turn,
        // 22.0 / 21.7; 512 x 7168 x 2048, rank 32, 15 mixed, 44.8 / 47.8, rank
        // 128, 2 in runs, 91.3 / 41.8, rank 16, 64 in turn, 40.0 / 81.9;
        // 700 x 1024, 4 mixed, K 4096, rank 16, 20.1 / 26.8, rank 64, 31.4 / 29.1;
        // 64 x 7168 x 2048, rank 64, 8 in turn, 22.1 / 39.2, rank 128, 2 in runs,
        // 23.4 / 18.5; 1024 x 7168 x 2048, rank 32, 64 in turn, 72 / 122, in
        // runs 76 / 55; 1024 x 1024 x 7168, rank 32, 8 in runs, 33.4 / 37.5.  K
        // below 1024 saves no more (64 x 7168 x 256, rank 32, 9.6 / 15.8).
        const int64_t work = M * N * R / std::max<int64_t>(K, 1024);
        few = (M <= 32 || (M <= 1536 && work <= 4096 * std::max<int64_t>(4, std::min<int64_t>(L, 32)))) &&
              N <= 65536 && K <= 65536;
        const int KB4 = (int)((K / 128 + 3) / 4);
        T = M <= 16 ? 1 : M <= 32 ? 2 : 4;
        row_tiles = few ? (int)((M + 16 * T - 1) / (16 * T)) : 0;
        col_tiles = few ? (int)((N + 127) / 128) : 0;
        const int want = few ? std::max(1, std::min(16, 256 / (row_tiles * col_tiles))) : 1;
        per = (KB4 + want - 1) / want * 4;
        shares = (KB4 * 4 + per - 1) / per;
        const int rows = 16 * (few ? 1 : R <= 64 ? 2 : 1);
        // Beyond a few row blocks, rows are grouped by adapter, so that one is
        // read once per block of its rows however they are mixed: the shrink of
        // 1455 rows of K 6400, 36 adapters of rank 16 in turn, 93 -> 10.3 us;
        // 4096 rows of K 2048, 8 packed prompts, rank 64, 12.4 -> 14.6 us.  One
        // adapter, or more ids than a workgroup looks through in a few
        // microseconds, are taken as they come.
        grouped = M > 64 && M <= 8192 && L > 1 && L <= 1024 && M * K < (int64_t(1) << 30);
        blocks = (M + rows - 1) / rows + (grouped ? std::min(L, M) : 0);
        // ungrouped, few row blocks take their adapters side by side; many have
        // the CUs' LDS to fill without workgroups that may find no adapter
        slots = few && !grouped ? (int)std::min<int64_t>(L, 16) : 1;
        // few row blocks give few workgroups, so K is split over more of them
        parts = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxParts, (few ? 64 : 256) / blocks, K / 256}));
        auto up = [](int64_t v) { return (v + 255) & ~int64_t(255); };
        low = 0;
        sums = up(parts * M * R * 4);
        total = sums + (few ? up((int64_t)shares * M * N * 4) : 0);
    }
};

int64_t lora_workspace(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    return M == 0 ? 0 : LoraPlan(M, N, K, L, R).total;
}

dg_status lora_limits(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    const LoraPlan at(M, N, K, L, R);
    if (at.few) return DG_OK;
    static_assert(ShrinkShape<1, true>::W == 8 && ShrinkShape<2, true>::W == 4 && ShrinkShape<4, true>::W == 4 &&
                      ShrinkShape<8, true>::W == 4,
                  "the shrink's workgroups");
    if (!grid_fits(at.blocks, R <= 16 ? 512 : 256)) return DG_ERR_SHAPE;
    GemmArgs d{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, M, N, K, 1, nullptr};
    d.check_only = true;
    return launch_gemm(Form::DenseLora, d, nullptr);
}

template <int RT>
static dg_status shrink(const ShrinkArgs& g, hipStream_t stream) {
    using Shape = ShrinkShape<RT, true>;
    hipLaunchKernelGGL((lora_shrink_kernel<RT>), dim3(g.blocks, g.slots, g.parts), dim3(64 * Shape::W),
                       Shape::kLds, stream, g);
    return launched();
}

template <int T, int RT, bool kE8>
static dg_status few(const FewArgs& f, const ShrinkArgs& g, hipStream_t stream) {
    constexpr size_t lds = std::max<size_t>(panel_lds<T, 1, kFewRing>(), ShrinkShape<RT, false>::kLds);
    const int grid = f.row_tiles * f.col_tiles * f.shares + g.blocks * g.slots * g.parts;
    hipLaunchKernelGGL((lora_few_kernel<T, RT, kE8>), dim3(grid), dim3(64 * kPanelWaves), lds, stream, f, g);
    return launched();
}

template <int RT, bool kE8>
static dg_status few_rows(const LoraPlan& at, const FewArgs& f, const ShrinkArgs& g, hipStream_t stream) {
    return at.T == 1   ? few<1, RT, kE8>(f, g, stream)
           : at.T == 2 ? few<2, RT, kE8>(f, g, stream)
                       : few<4, RT, kE8>(f, g, stream);
}

template <int RT, bool kE8>
static dg_status lora_rank(const LoraArgs& a, hipStream_t stream) {
    const LoraPlan at(a.M, a.N, a.K, a.L, a.R);
    uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
    float* const low = reinterpret_cast<float*>(ws + at.low);
    const ShrinkArgs g{a.x, a.lora_a, a.ids, low, a.M, a.K, a.L, a.R, (int)at.blocks, at.slots, at.parts, at.grouped};
    if (at.few) {
        float* const sums = reinterpret_cast<float*>(ws + at.sums);
        const FewArgs f{a.A, a.sa, a.B, a.sb, sums, (int)a.M, (int)a.N, (int)a.K, at.row_tiles, at.col_tiles,
                        at.shares, at.per};
        const dg_status s = few_rows<RT, kE8>(at, f, g, stream);
        if (s != DG_OK) return s;
        hipLaunchKernelGGL((lora_combine_kernel<2 * RT>), dim3((unsigned)((a.N + 255) / 256), (unsigned)a.M),
                           dim3(256), 0, stream, sums, low, a.lora_b, a.scaling, a.ids, a.D, (int)a.M, (int)a.N,
                           a.L, a.R, at.parts, at.shares);
        return launched();
    }
    const dg_status s = shrink<RT>(g, stream);
    if (s != DG_OK) return s;
    GemmArgs d{a.A, a.sa, a.B, a.sb, a.D, nullptr, a.M, a.N, a.K, 1, nullptr};
    d.e8m0 = kE8;
    d.lora = LoraTail{low, a.lora_b, a.scaling, a.ids, at.parts, a.L, a.R};
    return launch_gemm(Form::DenseLora, d, stream);
}

template <bool kE8>
static dg_status lora_scales(const LoraArgs& a, hipStream_t stream) {
    if (a.R <= 16) return lora_rank<1, kE8>(a, stream);
    if (a.R <= 32) return lora_rank<2, kE8>(a, stream);
    if (a.R <= 64) return lora_rank<4, kE8>(a, stream);
    return lora_rank<8, kE8>(a, stream);
}

dg_status launch_lora(const LoraArgs& a, bool e8m0, hipStream_t stream) {
    return e8m0 ? lora_scales<true>(a, stream) : lora_scales<false>(a, stream);
}

}  // namespace dg
