// The steps of an expert layer for many tokens around the grouped products.
// include/dg_experts.h has the definitions.
#include "experts_launch.h"

#include <algorithm>
#include <type_traits>

#include "dispatch_form.h"
#include "layout_share.h"
#include "rows_common.h"

namespace dg {

// ------------------------------------------------------------------ the sort
//
// A stable counting sort by expert, without atomics on memory: (1) each
// workgroup counts its run of pairs per expert into a table [run][E]; (2) each
// workgroup adds up the table's columns (all of it: the experts' sizes; the
// runs before its own: where its pairs go on), turns the sizes into padded
// offsets, and places its pairs 1024 at a time.  Within a wave a pair's rank is
// the number of lanes below it with the same expert, from one ballot per bit of
// the expert's number; across the 16 waves of a tile each wave leaves its count
// in a byte per expert, so that a pair's rank in the tile is a sum of at most 16
// bytes.  One run alone needs no table and one launch.

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
// Pairs that one workgroup sorts by itself: one tile.  256 experts: 1024 pairs 8.4
// us; 2048 pairs 9.8 in one workgroup, 9.7 in two and two launches, 8192 pairs
// 17.5 and 9.3.  16 experts: 2048 pairs 6.0 and 7.3, 8192 11.8 and 7.6.
constexpr int kSortOnePairs = 1024;
constexpr int kSortMaxRuns = 256;

// Pairs in a run, a multiple of the tile.
static int64_t sort_run(int64_t P) {
    if (P <= kSortOnePairs) return kSortOnePairs;
    return std::max<int64_t>(1024, ((P + kSortMaxRuns - 1) / kSortMaxRuns + 1023) / 1024 * 1024);
}
static int sort_runs(int64_t P) { return (int)std::max<int64_t>(1, (P + sort_run(P) - 1) / sort_run(P)); }

int64_t sort_workspace(int64_t T, int64_t k, int64_t E) {
    const int runs = sort_runs(T * k);
    return runs == 1 ? 0 : (int64_t)runs * E * 4;
}

// The number of pairs of each expert among ids [begin, end), added to count[E]
// in LDS by n threads; with kBefore also of those before pair `split`.  Eight
// loads at a time: one after the other each waits for memory.
template <bool kBefore>
__device__ __forceinline__ void count_pairs(const int32_t* __restrict__ ids, int64_t begin, int64_t end, int E,
                                            int* count, int tid, int n, int* before = nullptr, int64_t split = 0) {
    for (int64_t p0 = begin; p0 < end; p0 += 8 * n) {
        int e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t p = p0 + i * n + tid;
            e[i] = p < end ? ids[p] : -1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (e[i] < 0 || e[i] >= E) continue;
            atomicAdd(&count[e[i]], 1);
            if (kBefore && p0 + i * n + tid < split) atomicAdd(&before[e[i]], 1);
        }
    }
}

__global__ __launch_bounds__(kSortThreads) void moe_sort_count_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                                      int64_t run, int* __restrict__ table) {
    extern __shared__ int count[];
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += kSortThreads) count[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * run;
    count_pairs<false>(ids, begin, min(begin + run, P), E, count, tid, kSortThreads);
    __syncthreads();
    for (int e = tid; e < E; e += kSortThreads) table[(int64_t)blockIdx.x * E + e] = count[e];
}

// offsets[0 .. E] in LDS from the experts' sizes: each padded to 128, summed
// exclusively.  `part` holds a wave's sum each; all threads of the workgroup.
template <int kThreads>
__device__ __forceinline__ void padded_offsets(const int* size, int* offsets, int* part, int E, int tid) {
    const int each = (E + kThreads - 1) / kThreads, first = tid * each;
    int own = 0;
    for (int i = 0; i < each; ++i)
        if (first + i < E) own += (size[first + i] + 127) & ~127;
    int upto = own;  // over the wave's lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int below = __shfl_up(upto, d, 64);
        if ((tid & 63) >= d) upto += below;
    }
    if ((tid & 63) == 63) part[tid >> 6] = upto;
    __syncthreads();
    int at = upto - own;
    for (int w = 0; w < (tid >> 6); ++w) at += part[w];
    for (int i = 0; i < each; ++i)
        if (first + i < E) {
            offsets[first + i] = at;
            at += (size[first + i] + 127) & ~127;
            if (first + i == E - 1) offsets[E] = at;
        }
    __syncthreads();
}

// The expert whose rows, or padding, hold sorted row r < offsets[E]: the last
// one that starts at or before it (one without rows starts where the next does).
__device__ __forceinline__ int expert_of(const int* offsets, int E, int r) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (offsets[mid] <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The number of lanes below this one whose bit is set.
__device__ __forceinline__ int lanes_below(uint64_t bits) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(bits >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)bits, 0));
}

// layout of M rows, by `waves` waves (at most kLayoutWaves) of which this is the
// `wave`-th, from the experts' offsets and sizes (LDS): the experts that have
// pairs are dealt out to the waves, several to an expert's blocks where there
// are more waves than experts, and then the rows behind the last expert's.  (A
// search for each block's expert took 10 of 15 us where one workgroup sorts 512
// pairs of 256 experts.)
__device__ __forceinline__ void write_layout(const int* offsets, const int* size, int E, int64_t M, int wave, int waves,
                                             int32_t* __restrict__ layout, int lane) {
    auto blocks = [&](int e, int begin, int step) {
        const int first = offsets[e], n = size[e];
        each_block(n, begin, step, [&](int r) {
            const int at = r + 2 * lane;
            *reinterpret_cast<int2*>(layout + first + at) = int2{at < n ? e : -1, at + 1 < n ? e : -1};
        });
    };
    if (waves > E) {
        const BlockShare s = block_share(wave, waves, E);
        blocks(s.expert, s.begin, s.step);
    } else {
        int before = 0;  // used experts in front of e0
        for (int e0 = 0; e0 < E; e0 += 64) {
            const bool has = e0 + lane < E && size[min(e0 + lane, E - 1)] > 0;
            const uint64_t used = __ballot(has);
            uint64_t mine = __ballot(has && (before + lanes_below(used)) % waves == wave);
            for (; mine != 0; mine &= mine - 1) blocks(e0 + __builtin_ctzll(mine), 0, 1);
            before += __popcll(used);
        }
    }
    each_rest(offsets[E], M, wave, waves, lane,
              [&](int64_t r) { *reinterpret_cast<int4*>(layout + r) = int4{-1, -1, -1, -1}; });
}

// Sum over 16 byte counts of one expert: those of the waves before `wave`, and
// of all of them.
__device__ __forceinline__ void sum_counts(const v4u& c, int wave, int& before, int& all) {
    uint32_t b = 0, s = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int bytes = min(max(wave - 4 * w, 0), 4);
        const uint32_t mask = bytes == 4 ? 0xffffffffu : (1u << (8 * bytes)) - 1u;
        b = __builtin_amdgcn_sad_u8(c[w] & mask, 0, b);
        s = __builtin_amdgcn_sad_u8(c[w], 0, s);
    }
    before = (int)b;
    all = (int)s;
}

static size_t sort_lds(int E) { return (size_t)E * 16 + (size_t)E * 4 * 2 + (size_t)(E + 1) * 4 + kSortWaves * 4 + 16; }

__global__ __launch_bounds__(kSortThreads) void moe_sort_place_kernel(const int32_t* __restrict__ ids, int64_t P, int E,
                                                                      int64_t run, int runs,
                                                                      const int* __restrict__ table,
                                                                      int32_t* __restrict__ rows,
                                                                      int32_t* __restrict__ layout,
                                                                      int32_t* __restrict__ out_offsets, int64_t M) {
    extern __shared__ __align__(16) uint8_t lds[];
    v4u* const counts = reinterpret_cast<v4u*>(lds);         // [E] a byte for each wave
    int* const size = reinterpret_cast<int*>(counts + E);    // [E]
    int* const next = size + E;                              // [E] row of the next pair
    int* const offsets = next + E;                           // [E + 1]
    int* const part = offsets + E + 1;                       // [kSortWaves]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int me = blockIdx.x;
    const int64_t begin = me * run, end = min(begin + run, P);
    int id = begin + tid < end ? ids[begin + tid] : -1;  // of the tile that is placed next
    for (int e = tid; e < E; e += kSortThreads) {
        counts[e] = v4u{0, 0, 0, 0};
        size[e] = next[e] = 0;
    }
    __syncthreads();
    if (runs == 1) {
        count_pairs<false>(ids, 0, P, E, size, tid, kSortThreads);
    } else {
        // the table's rows shared out over groups of threads where experts are few
        int width = 64;
        while (width < E && width < kSortThreads) width *= 2;
        const int group = tid / width, groups = kSortThreads / width;
        for (int e = tid % width; e < E; e += width) {
            int all = 0, before = 0;
            for (int r0 = group; r0 < runs; r0 += 8 * groups) {
                int n[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] = table[(int64_t)min(r0 + i * groups, runs - 1) * E + e];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (r0 + i * groups < runs) all += n[i];
                    if (r0 + i * groups < me) before += n[i];
                }
            }
            atomicAdd(&size[e], all);
            atomicAdd(&next[e], before);
        }
    }
    __syncthreads();
    padded_offsets<kSortThreads>(size, offsets, part, E, tid);
    for (int e = tid; e < E; e += kSortThreads) next[e] += offsets[e];
    if (me == 0)
        for (int e = tid; e <= E; e += kSortThreads) out_offsets[e] = offsets[e];
    __syncthreads();

    const int bits = 32 - __builtin_clz(max(E - 1, 1));
    for (int64_t base = begin; base < end; base += kSortThreads) {
        const int64_t p = base + tid;
        const int e = id;
        id = p + kSortThreads < end ? ids[p + kSortThreads] : -1;
        const bool here = e >= 0 && e < E;
        uint64_t same = __ballot(here);
        for (int b = 0; b < bits; ++b) {
            const bool bit = (e >> b) & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const int rank = lanes_below(same);
        if (here && rank == 0) reinterpret_cast<uint8_t*>(counts + e)[wave] = (uint8_t)__popcll(same);
        __syncthreads();
        int before = 0, all = 0;
        if (here) {
            sum_counts(counts[e], wave, before, all);
            rows[p] = next[e] + before + rank;
        } else if (p < end) {
            rows[p] = -1;
        }
        if (base + kSortThreads < end) {
            __syncthreads();
            if (here && before == 0 && rank == 0) {  // one pair of each expert in the tile
                next[e] += all;
                counts[e] = v4u{0, 0, 0, 0};
            }
            __syncthreads();
        }
    }
    write_layout(offsets, size, E, M, me * kSortWaves + wave, runs * kSortWaves, layout, lane);
}

dg_status launch_sort(const SortArgs& a, hipStream_t stream) {
    const int64_t P = a.T * a.k, run = sort_run(P);
    const int runs = sort_runs(P);
    int* const table = static_cast<int*>(a.workspace);
    if (runs > 1) {
        hipLaunchKernelGGL(moe_sort_count_kernel, dim3(runs), dim3(kSortThreads), a.E * 4, stream, a.ids, P, a.E, run,
                           table);
        if (launched() != DG_OK) return DG_ERR_HIP;
    }
    hipLaunchKernelGGL(moe_sort_place_kernel, dim3(runs), dim3(kSortThreads), sort_lds(a.E), stream, a.ids, P, a.E, run,
                       runs, table, a.rows, a.layout, a.offsets, a.M);
    return launched();
}

// --------------------------------------------------------------- the copies

// Sets rows to zero: those of the kZeroRows from r0 on whose bit is set.
__device__ __forceinline__ void zero_rows(uint16_t* __restrict__ out, int64_t r0, uint64_t which, int64_t H, int tid) {
    for (; which != 0; which &= which - 1) {
        uint16_t* const row = out + (r0 + __builtin_ctzll(which)) * H;
        for (int64_t c = tid; c < H / 8; c += 256) *reinterpret_cast<v4u*>(row + c * 8) = v4u{0, 0, 0, 0};
    }
}

// The same for those whose layout entry is negative; every lane looks at one.
__device__ __forceinline__ void zero_padding(uint16_t* __restrict__ out, const int32_t* __restrict__ layout, int64_t M,
                                             int64_t H, int64_t group, int tid) {
    const int64_t r0 = group * kZeroRows, r = r0 + (tid & 63);
    const bool pad = (tid & 63) < kZeroRows && r < M && layout[r] < 0;
    zero_rows(out, r0, __ballot(pad), H, tid);
}

// Where a copy finds its tokens' rows: in memory, behind a sort of its own
// launches, or, for few pairs (dispatch_form.h), from a sort that every workgroup
// does for itself: it counts all pairs per expert, and those before its token's.
struct SmallSort {
    const int32_t* ids;
    int32_t *rows, *layout, *offsets;  // the plan's outputs
    int64_t M;
    int P, k, E;
};
constexpr int kMaxChoices = 64;

static size_t small_lds(int E) { return (size_t)(3 * E + 1) * 4; }

// Sorts for token t: row[0 .. k) in LDS, and the experts' offsets and sizes,
// which the caller's LDS at `lds` holds.  All 256 threads of the workgroup.
__device__ __forceinline__ void sort_token(const SmallSort& p, int64_t t, int* lds, int* part, int* row, int tid) {
    int* const size = lds;
    int* const before = size + p.E;
    int* const offsets = before + p.E;
    for (int e = tid; e < 2 * p.E; e += 256) size[e] = 0;
    __syncthreads();
    const int first = (int)(t * p.k);
    const int own = tid < p.k && first + tid < p.P ? p.ids[first + tid] : -1;
    count_pairs<true>(p.ids, 0, p.P, p.E, size, tid, 256, before, first);
    __syncthreads();
    padded_offsets<256>(size, offsets, part, p.E, tid);
    if (tid < 64) {  // the first wave, a lane for each choice
        const bool here = own >= 0 && own < p.E;
        int r = here ? offsets[own] + before[own] : -1;
        for (int j = 0; j < p.k; ++j) r += here && j < tid && __builtin_amdgcn_readlane(own, j) == own;
        if (tid < p.k) row[tid] = r;
    }
    __syncthreads();
}

// The plan's outputs, shared out over the copies' workgroups.
__device__ __forceinline__ void write_plan(const SmallSort& p, int64_t t, bool first_part, const int* lds, const int* row,
                                           int tid) {
    const int* const size = lds;
    const int* const offsets = size + 2 * p.E;
    if (first_part && tid < p.k && t * p.k + tid < p.P) p.rows[t * p.k + tid] = row[tid];
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int e = tid; e <= p.E; e += 256) p.offsets[e] = offsets[e];
    const unsigned wg = blockIdx.y * gridDim.x + blockIdx.x;  // of at most 2^24
    const int waves = layout_waves(gridDim.x * gridDim.y, 4), wave = (int)(wg * 4 + (tid >> 6));
    if (wave < waves) write_layout(offsets, size, p.E, p.M, wave, waves, p.layout, tid & 63);
}

// bf16 rows: a thread copies 8 columns of a token into each of its rows.  The
// grid's columns are parts of a token in the small form, all of the copies
// otherwise, and behind them workgroups that clear padding (in the small form
// they sort for themselves too).
template <bool kSmall>
__global__ __launch_bounds__(256) void moe_copy_bf16_kernel(const uint16_t* __restrict__ x,
                                                            const int32_t* __restrict__ rows,
                                                            const int32_t* __restrict__ layout,
                                                            uint16_t* __restrict__ out, int64_t T, int k, int64_t H,
                                                            int64_t M, unsigned copies, unsigned parts, SmallSort plan) {
    const int tid = threadIdx.x;
    const int64_t width = H / 8;
    if constexpr (kSmall) {
        extern __shared__ int plan_lds[];
        __shared__ int part[4], row[kMaxChoices];
        const int64_t t = blockIdx.x < copies ? blockIdx.x / parts : T;  // T: none, all pairs lie before it
        sort_token(plan, t, plan_lds, part, row, tid);
        if (t == T) {
            write_plan(plan, t, false, plan_lds, row, tid);
            const int* const size = plan_lds;
            const int* const offsets = size + 2 * plan.E;
            const int64_t r0 = (int64_t)(blockIdx.x - copies) * kZeroRows;
            const int64_t r = r0 + (tid & 63);
            bool pad = (tid & 63) < kZeroRows && r < M;
            if (pad && r < offsets[plan.E]) {
                const int e = expert_of(offsets, plan.E, (int)r);
                pad = r - offsets[e] >= size[e];
            }
            return zero_rows(out, r0, __ballot(pad), H, tid);
        }
        const int64_t c = blockIdx.x % parts * 256 + tid;
        if (c < width) {
            const v4u v = *reinterpret_cast<const v4u*>(x + t * H + c * 8);
            for (int j = 0; j < k; ++j)
                if (row[j] >= 0) *reinterpret_cast<v4u*>(out + row[j] * H + c * 8) = v;
        }
        write_plan(plan, t, blockIdx.x % parts == 0, plan_lds, row, tid);
    } else {
        if (blockIdx.x >= copies) return zero_padding(out, layout, M, H, blockIdx.x - copies, tid);
        const int64_t i = (int64_t)blockIdx.x * 256 + tid;
        if (i >= T * width) return;
        const int64_t t = i / width, c = i - t * width;
        const v4u v = *reinterpret_cast<const v4u*>(x + i * 8);
        for (int j = 0; j < k; ++j) {
            const int r = rows[t * k + j];
            if (r >= 0) *reinterpret_cast<v4u*>(out + r * H + c * 8) = v;
        }
    }
}

// Workgroup b of a grid, in an order that gives each of the 8 XCDs (b % 8) one
// run of them.
__device__ __forceinline__ int64_t xcd_run(unsigned b, unsigned grid) {
    const unsigned x = b % 8, per = grid / 8, more = grid % 8;
    return (int64_t)x * per + min(x, more) + b / 8;
}

// FP8 rows: eight lanes own one 128-column block of a token, as in the
// quantizer, and store its line of codes into each of the token's rows.  Bound
// by the stores: 4096 tokens of 7168 into 8 rows each, 243 MB, 64 us, 4.7 TB/s
// with the reads.  The scales of the workgroup's 32 blocks go out together and
// tokens in runs per XCD, so that rows beside each other meet in one L2 (76 us
// with the sort, 78 before, 71 without scales); a wave for each whole row took
// as long, stores past the caches too.
template <bool kE8, bool kSmall>
__global__ __launch_bounds__(256) void moe_copy_fp8_kernel(const uint16_t* __restrict__ x,
                                                           const int32_t* __restrict__ rows, uint8_t* __restrict__ q,
                                                           void* __restrict__ s, int64_t T, int k, int64_t H,
                                                           SmallSort plan) {
    using S = typename std::conditional<kE8, uint8_t, float>::type;
    __shared__ __align__(16) uint8_t lines[32][128];
    __shared__ S scales[32];
    __shared__ int part[kSmall ? 4 : 1], row[kSmall ? kMaxChoices : 1];
    extern __shared__ int plan_lds[];
    const int64_t KB = H >> 7;
    const int tid = threadIdx.x, group = tid >> 3, lane = tid & 7;
    const int64_t pitch = kE8 ? (KB + 3) & ~int64_t(3) : KB;
    // token and block of a group
    auto place = [&](int g, int64_t& t, int64_t& kb) __attribute__((always_inline)) {
        if constexpr (kSmall) {
            t = blockIdx.x;
            kb = (int64_t)blockIdx.y * 32 + g;
            return kb < KB;
        } else {
            const int64_t blk = xcd_run(blockIdx.x, gridDim.x) * 32 + g;
            t = blk / KB;
            kb = blk - t * KB;
            return blk < T * KB;
        }
    };
    auto target = [&](int64_t t, int j) __attribute__((always_inline)) -> int64_t {
        if constexpr (kSmall)
            return row[j];
        else
            return rows[t * k + j];
    };
    int64_t t, kb;
    const bool here = place(group, t, kb);
    v4u raw[2] = {};
    if (here) {
#pragma unroll
        for (int h = 0; h < 2; ++h) raw[h] = *reinterpret_cast<const v4u*>(x + t * H + kb * 128 + 64 * h + 8 * lane);
    }
    if constexpr (kSmall) sort_token(plan, t, plan_lds, part, row, tid);
    if (here) {
        float f[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) unpack_bf16(raw[h], f[h]);
        const auto scale = block_codes<kE8>(f, lines[group], lane);
        if (lane == 0) scales[group] = (S)scale;
        const v4u codes = *reinterpret_cast<const v4u*>(&lines[group][16 * lane]);
        for (int j = 0; j < k; ++j) {
            const int64_t r = target(t, j);
            if (r >= 0) *reinterpret_cast<v4u*>(q + r * H + kb * 128 + 16 * lane) = codes;
        }
    }
    __syncthreads();
    if (place(tid & 31, t, kb))
        for (int j = tid >> 5; j < k; j += 8) {
            const int64_t r = target(t, j);
            if (r >= 0) static_cast<S*>(s)[r * pitch + kb] = scales[tid & 31];
        }
    if constexpr (kSmall) write_plan(plan, blockIdx.x, blockIdx.y == 0, plan_lds, row, tid);
}

// int8 rows: one workgroup per token, as the scale needs all of it.  4096 tokens
// of 7168 into 8 rows each: 55 us, 5.4 TB/s; 66 with the sort of 256 experts.
template <int C, bool kSmall>
__global__ __launch_bounds__(256) void moe_copy_int8_kernel(const uint16_t* __restrict__ x,
                                                            const int32_t* __restrict__ rows, uint8_t* __restrict__ q,
                                                            float* __restrict__ s, int k, int64_t H, SmallSort plan) {
    __shared__ uint32_t tops[4];
    __shared__ int part[4], row[kMaxChoices];
    extern __shared__ int plan_lds[];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    if constexpr (kSmall) {
        sort_token(plan, t, plan_lds, part, row, tid);
    } else {
        if (tid < k) row[tid] = rows[t * k + tid];
    }
    // the barrier inside is in front of the first store
    const float scale = int8_row<256, C>(
        H / 8, tid, tops,
        [&](int64_t c, float (&f)[8]) { unpack_bf16(*reinterpret_cast<const v4u*>(x + t * H + c * 8), f); },
        [&](int64_t c, const v2u& codes) {
            for (int j = 0; j < k; ++j)
                if (row[j] >= 0) *reinterpret_cast<v2u*>(q + row[j] * H + c * 8) = codes;
        });
    if (tid < k && row[tid] >= 0) s[row[tid]] = scale;
    if constexpr (kSmall) write_plan(plan, t, true, plan_lds, row, tid);
}

static int64_t zero_grid(int64_t M, Held held) { return held == Held::Bf16 ? (M + kZeroRows - 1) / kZeroRows : 0; }

static int64_t copy_grid(int64_t T, int64_t H, Held held) {
    switch (held) {
        case Held::Bf16: return (T * (H / 8) + 255) / 256;
        case Held::Int8: return T;
        default: return (T * (H >> 7) + 31) / 32;
    }
}

static bool small_sort(int64_t T, int64_t k, int64_t E, int64_t H, int64_t M, Held held) {
    return sorts_for_itself(T * k, E,
                            held == Held::Bf16   ? small_grid_bf16(T, H, M)
                            : held == Held::Int8 ? T
                                                 : small_grid_fp8(T, H));
}

dg_status dispatch_limits(int64_t T, int64_t k, int64_t E, int64_t H, int64_t M, Held held) {
    if (small_sort(T, k, E, H, M, held)) return DG_OK;  // at most kSmallSteps / 4 workgroups
    return grid_fits(copy_grid(T, H, held) + zero_grid(M, held), 256) ? DG_OK : DG_ERR_SHAPE;
}

template <bool kSmall>
static dg_status launch_copies(const DispatchArgs& a, Held held, hipStream_t stream) {
    const SortArgs& p = a.sort;
    const SmallSort plan{p.ids, p.rows, p.layout, p.offsets, p.M, (int)(kSmall ? p.T * p.k : 0), p.k, p.E};
    const size_t lds = kSmall ? small_lds(p.E) : 0;
    const dim3 block(256);
    uint8_t* const q = static_cast<uint8_t*>(a.out);
    const int64_t zero = zero_grid(p.M, held);
    if (held == Held::Bf16) {
        const int64_t parts = (a.H / 8 + 255) / 256;
        const int64_t copies = kSmall ? p.T * parts : copy_grid(p.T, a.H, held);
        if (copies + zero == 0) return DG_OK;
        hipLaunchKernelGGL(moe_copy_bf16_kernel<kSmall>, dim3((unsigned)(copies + zero)), block, lds, stream, a.x, p.rows,
                           p.layout, static_cast<uint16_t*>(a.out), p.T, p.k, a.H, p.M, (unsigned)copies,
                           (unsigned)parts, plan);
        return launched();
    }
    if (p.T == 0) return DG_OK;
    if (held == Held::Int8) {
        auto kernel = a.H <= 8192 ? moe_copy_int8_kernel<4, kSmall> : moe_copy_int8_kernel<0, kSmall>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)p.T), block, lds, stream, a.x, p.rows, q, static_cast<float*>(a.s), p.k,
                           a.H, plan);
        return launched();
    }
    const dim3 grid = kSmall ? dim3((unsigned)p.T, (unsigned)(((a.H >> 7) + 31) / 32))
                             : dim3((unsigned)copy_grid(p.T, a.H, held));
    if (held == Held::Fp8)
        hipLaunchKernelGGL((moe_copy_fp8_kernel<false, kSmall>), grid, block, lds, stream, a.x, p.rows, q, a.s, p.T, p.k,
                           a.H, plan);
    else
        hipLaunchKernelGGL((moe_copy_fp8_kernel<true, kSmall>), grid, block, lds, stream, a.x, p.rows, q, a.s, p.T, p.k,
                           a.H, plan);
    return launched();
}

dg_status launch_dispatch(const DispatchArgs& a, Held held, hipStream_t stream) {
    const SortArgs& p = a.sort;
    if (small_sort(p.T, p.k, p.E, a.H, p.M, held)) return launch_copies<true>(a, held, stream);
    const dg_status st = launch_sort(p, stream);
    return st != DG_OK ? st : launch_copies<false>(a, held, stream);
}

// ------------------------------------------------------- the weighted sum back

// A thread adds up 8 columns of a token, eight of its rows in flight at once;
// entries without a row load row 0 for nothing, which costs less than a branch
// around each load (4096 tokens of 8 rows of 7168: 104 us against 106, 5.1 TB/s;
// 61 tokens of 6: 3.3 against 3.8).  More tokens an XCD in a row (109 us) or
// fewer workgroups a CU (102) changed little.
__global__ __launch_bounds__(256) void moe_unpermute_kernel(const uint16_t* __restrict__ y,
                                                            const int32_t* __restrict__ rows,
                                                            const float* __restrict__ weights,
                                                            uint16_t* __restrict__ out, int64_t T, int k, int64_t H,
                                                            int64_t M) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, width = H / 8;
    if (i >= T * width) return;
    const int64_t t = i / width, c = i - t * width;
    float sum[8] = {};
    for (int j0 = 0; j0 < k; j0 += 8) {
        v4u v[8];
        float w[8];
        bool on[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = j0 + j < k ? rows[t * k + j0 + j] : -1;
            w[j] = weights != nullptr && j0 + j < k ? weights[t * k + j0 + j] : 1.0f;
            on[j] = r >= 0 && r < M;
            v[j] = *reinterpret_cast<const v4u*>(y + (on[j] ? r : 0) * H + c * 8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f[8];
            unpack_bf16(v[j], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = on[j] ? __builtin_fmaf(w[j], f[e], sum[e]) : sum[e];
        }
    }
    *reinterpret_cast<v4u*>(out + i * 8) = pack_bf16(sum);
}

dg_status launch_unpermute(const UnpermuteArgs& a, hipStream_t stream) {
    const int64_t grid = (a.T * (a.H / 8) + 255) / 256;
    if (!grid_fits(grid, 256)) return DG_ERR_SHAPE;
    // without sorted rows there is no row 0 either: no choices, zeros
    hipLaunchKernelGGL(moe_unpermute_kernel, dim3((unsigned)grid), dim3(256), 0, stream, a.y, a.rows, a.weights, a.out,
                       a.T, a.M > 0 ? a.k : 0, a.H, a.M);
    return launched();
}

// One workgroup per token and eight of its choices at a time: a thread holds
// its columns of the gradient, scales them into each row's gradient and keeps
// the eight dot products, so that both gradients take one pass.  The workgroups
// behind the tokens clear padding.  Bound by memory: 4096 tokens of 8 rows of
// 7168, 1.0 GB, in 206 us (4.8 TB/s), and 0.47 GB of zeros in 85; rows cleared
// one, 4 or 16 to a workgroup, first or last, and other workgroup sizes are
// within 2% of each other.
__global__ __launch_bounds__(256) void moe_unpermute_backward_kernel(
    const uint16_t* __restrict__ grad, const uint16_t* __restrict__ y, const int32_t* __restrict__ rows,
    const float* __restrict__ weights, const int32_t* __restrict__ layout, uint16_t* __restrict__ grad_y,
    float* __restrict__ grad_weights, int64_t T, int k, int64_t H, int64_t M) {
    __shared__ float parts[4][8];
    const int tid = threadIdx.x;
    if (blockIdx.x >= T) return zero_padding(grad_y, layout, M, H, blockIdx.x - T, tid);
    const int64_t t = blockIdx.x;
    for (int j0 = 0; j0 < k; j0 += 8) {
        int64_t r[8];
        float w[8], dot[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = j0 + j < k ? rows[t * k + j0 + j] : -1;
            if (r[j] >= M) r[j] = -1;
            w[j] = r[j] >= 0 && weights != nullptr ? weights[t * k + j0 + j] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int64_t c = tid; c < H / 8; c += 256) {
            float g[8];
            unpack_bf16(*reinterpret_cast<const v4u*>(grad + t * H + c * 8), g);
            v4u v[8];
            if (grad_weights != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (r[j] >= 0) v[j] = *reinterpret_cast<const v4u*>(y + r[j] * H + c * 8);
            }
            if (grad_y != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (r[j] < 0) continue;
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] = w[j] * g[e];
                    *reinterpret_cast<v4u*>(grad_y + r[j] * H + c * 8) = pack_bf16(d);
                }
            }
            if (grad_weights != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (r[j] < 0) continue;
                    float f[8];
                    unpack_bf16(v[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] = __builtin_fmaf(g[e], f[e], dot[j]);
                }
            }
        }
        if (grad_weights != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float sum = wave_sum(dot[j]);
                if ((tid & 63) == 0) parts[tid >> 6][j] = sum;
            }
            __syncthreads();
            if (tid < 8 && j0 + tid < k)
                grad_weights[t * k + j0 + tid] = (parts[0][tid] + parts[1][tid]) + (parts[2][tid] + parts[3][tid]);
            __syncthreads();
        }
    }
}

dg_status launch_unpermute_backward(const UnpermuteBackwardArgs& a, hipStream_t stream) {
    const int64_t zero = a.grad_y != nullptr && a.layout != nullptr ? (a.M + kZeroRows - 1) / kZeroRows : 0;
    if (a.T + zero == 0) return DG_OK;
    if (!grid_fits(a.T + zero, 256)) return DG_ERR_SHAPE;
    hipLaunchKernelGGL(moe_unpermute_backward_kernel, dim3((unsigned)(a.T + zero)), dim3(256), 0, stream, a.grad, a.y,
                       a.rows, a.weights, a.layout, a.grad_y, a.grad_weights, a.T, a.k, a.H, a.M);
    return launched();
}

// ------------------------------------------------------------------ the gate

// sigmoid(g) for a bf16 g, off by at most 5 * 2^-24 of itself where it is 2^-126
// or more (g above -87.3), by less than 2^-126 below that, where it may come as 0:
// the reciprocal has no subnormal results, and 1 + exp(-g) is infinite from 2^128 on.
// exp(-g) is 2^n 2^f with n the integer nearest to -g log2(e), and f, at most
// 1/2, from two fused steps (g has 8 bits and the upper part of log2(e) 16, so
// that -g hi - n is exact); then the hardware's 2^f and reciprocal (an ulp
// each).  With the library's exponential and a full division the arithmetic, not
// memory, bounded the gate (32768 rows of 2048 in 95 us, 57 at a copy's rate).
__device__ __forceinline__ float sigmoid_bf16(float g) {
    constexpr float kHi = 1.44268798828125f;          // log2(e), 16 bits
    constexpr float kLo = (float)(1.4426950408889634 - 1.44268798828125);
    const float x = __builtin_amdgcn_fmed3f(-g, -200.0f, 200.0f);  // past which it is 0 or 1; keeps infinities out of f
    const float n = __builtin_rintf(x * (kHi + kLo));
    const float f = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -n));
    const float e = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// silu(gate) * up of eight columns.
__device__ __forceinline__ void gate8(const uint16_t* __restrict__ z, int64_t I, float (&h)[8]) {
    float g[8], u[8];
    unpack_bf16(*reinterpret_cast<const v4u*>(z), g);
    unpack_bf16(*reinterpret_cast<const v4u*>(z + I), u);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = g[e] * sigmoid_bf16(g[e]) * u[e];
}

__global__ __launch_bounds__(256) void swiglu_bf16_kernel(const uint16_t* __restrict__ z,
                                                          const int32_t* __restrict__ layout,
                                                          uint16_t* __restrict__ h, int64_t M, int64_t I) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, width = I / 8;
    if (i >= M * width) return;
    const int64_t r = i / width, c = i - r * width;
    v4u v = {0, 0, 0, 0};
    if (layout == nullptr || layout[r] >= 0) {
        float f[8];
        gate8(z + r * 2 * I + c * 8, I, f);
        v = pack_bf16(f);
    }
    *reinterpret_cast<v4u*>(h + i * 8) = v;
}

// Eight lanes per 128-column block of a row, as in the quantizer.  32768 rows of
// 2048 among 65280: 68 us, 4.9 TB/s.
template <bool kE8>
__global__ __launch_bounds__(256) void swiglu_fp8_kernel(const uint16_t* __restrict__ z,
                                                         const int32_t* __restrict__ layout, uint8_t* __restrict__ q,
                                                         void* __restrict__ s, int64_t M, int64_t I) {
    __shared__ __align__(16) uint8_t lines[32][128];
    const int64_t KB = I >> 7;
    const int group = threadIdx.x >> 3, lane = threadIdx.x & 7;
    const int64_t blk = (int64_t)blockIdx.x * 32 + group;
    if (blk >= M * KB) return;  // uniform over each 8-lane group, as is the next
    const int64_t r = blk / KB, kb = blk - r * KB;
    if (layout != nullptr && layout[r] < 0) return;
    float f[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) gate8(z + r * 2 * I + kb * 128 + 64 * h + 8 * lane, I, f[h]);
    const auto scale = block_codes<kE8>(f, lines[group], lane);
    *reinterpret_cast<v4u*>(q + blk * 128 + 16 * lane) = *reinterpret_cast<const v4u*>(&lines[group][16 * lane]);
    if (lane == 0) {
        if constexpr (kE8)
            static_cast<uint8_t*>(s)[r * ((KB + 3) & ~int64_t(3)) + kb] = (uint8_t)scale;
        else
            static_cast<float*>(s)[blk] = scale;
    }
}

// A row by G threads, as the scale needs all of it.  32768 rows of 2048: 71 us,
// 4.7 TB/s (88 by a workgroup each that computes the gate twice).
template <int G, int C>
__global__ __launch_bounds__(256) void swiglu_int8_kernel(const uint16_t* __restrict__ z,
                                                          const int32_t* __restrict__ layout, uint8_t* __restrict__ q,
                                                          float* __restrict__ s, int64_t M, int64_t I) {
    __shared__ uint32_t tops[4];
    const int64_t r = blockIdx.x * (int64_t)(256 / G) + threadIdx.x / G;
    if (r >= M || (layout != nullptr && layout[r] < 0)) return;  // uniform over the row's threads
    const int id = threadIdx.x % G;
    const float scale = int8_row<G, C>(
        I / 8, id, tops, [&](int64_t c, float (&f)[8]) { gate8(z + r * 2 * I + c * 8, I, f); },
        [&](int64_t c, const v2u& codes) { *reinterpret_cast<v2u*>(q + r * I + c * 8) = codes; });
    if (id == 0) s[r] = scale;
}

// Rows of up to 512 or 2048 columns by a wave each, wider ones by a workgroup.
static int64_t int8_rows_grid(int64_t M, int64_t width) { return width <= 256 ? (M + 3) / 4 : M; }

dg_status launch_swiglu(const SwigluArgs& a, Held held, hipStream_t stream) {
    const int64_t grid = held == Held::Bf16   ? (a.M * (a.I / 8) + 255) / 256
                         : held == Held::Int8 ? int8_rows_grid(a.M, a.I / 8)
                                              : (a.M * (a.I >> 7) + 31) / 32;
    if (!grid_fits(grid, 256)) return DG_ERR_SHAPE;
    const dim3 blocks((unsigned)grid), threads(256);
    uint8_t* const q = static_cast<uint8_t*>(a.out);
    switch (held) {
        case Held::Bf16:
            hipLaunchKernelGGL(swiglu_bf16_kernel, blocks, threads, 0, stream, a.z, a.layout,
                               static_cast<uint16_t*>(a.out), a.M, a.I);
            break;
        case Held::Fp8:
            hipLaunchKernelGGL(swiglu_fp8_kernel<false>, blocks, threads, 0, stream, a.z, a.layout, q, a.s, a.M, a.I);
            break;
        case Held::Fp8E8:
            hipLaunchKernelGGL(swiglu_fp8_kernel<true>, blocks, threads, 0, stream, a.z, a.layout, q, a.s, a.M, a.I);
            break;
        case Held::Int8:
            hipLaunchKernelGGL(a.I <= 512    ? (swiglu_int8_kernel<64, 1>)
                               : a.I <= 2048 ? (swiglu_int8_kernel<64, 4>)
                               : a.I <= 8192 ? (swiglu_int8_kernel<256, 4>)
                                             : (swiglu_int8_kernel<256, 0>),
                               blocks, threads, 0, stream, a.z, a.layout, q, static_cast<float*>(a.s), a.M, a.I);
            break;
    }
    return launched();
}

// Both gradients of eight columns, from the gate recomputed.  4096 rows of 1408
// among 18304: 19 us, 58 MB and 80 MB of zeros.
__global__ __launch_bounds__(256) void swiglu_backward_kernel(const uint16_t* __restrict__ z,
                                                              const uint16_t* __restrict__ grad_h,
                                                              const int32_t* __restrict__ layout,
                                                              uint16_t* __restrict__ grad_z, int64_t M, int64_t I) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, width = I / 8;
    if (i >= M * width) return;
    const int64_t r = i / width, c = i - r * width, at = r * 2 * I + c * 8;
    v4u to_g = {0, 0, 0, 0}, to_u = {0, 0, 0, 0};
    if (layout == nullptr || layout[r] >= 0) {
        float g[8], u[8], d[8];
        unpack_bf16(*reinterpret_cast<const v4u*>(z + at), g);
        unpack_bf16(*reinterpret_cast<const v4u*>(z + at + I), u);
        unpack_bf16(*reinterpret_cast<const v4u*>(grad_h + i * 8), d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float p = sigmoid_bf16(g[e]), silu = g[e] * p;
            const float slope = p * (1.0f + g[e] * (1.0f - p));
            g[e] = d[e] * u[e] * slope;
            u[e] = d[e] * silu;
        }
        to_g = pack_bf16(g);
        to_u = pack_bf16(u);
    }
    *reinterpret_cast<v4u*>(grad_z + at) = to_g;
    *reinterpret_cast<v4u*>(grad_z + at + I) = to_u;
}

dg_status launch_swiglu_backward(const SwigluBackwardArgs& a, hipStream_t stream) {
    const int64_t grid = (a.M * (a.I / 8) + 255) / 256;
    if (!grid_fits(grid, 256)) return DG_ERR_SHAPE;
    hipLaunchKernelGGL(swiglu_backward_kernel, dim3((unsigned)grid), dim3(256), 0, stream, a.z, a.grad_h, a.layout,
                       a.grad_z, a.M, a.I);
    return launched();
}

}  // namespace dg
