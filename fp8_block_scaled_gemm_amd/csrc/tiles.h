// Output tiles of the products: their shapes, how workgroups map to them, and
// which rows of a 128-row block belong to one group.
#pragma once

#include <atomic>

#include "device_common.h"
#include "tile_order.h"
#include "wave_ops.h"

namespace dg {

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int GROUP_M_>
struct TileConfig {
    static constexpr int BM = BM_, BN = BN_;
    static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
    static constexpr int kWaves = WAVES_M * WAVES_N;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;  // rows / cols per wave
    static constexpr int TM = WM / 16, TN = WN / 16;            // 16x16 sub-tiles per wave
    static constexpr int kGroupM = GROUP_M_;                    // m-blocks per raster group
    // one wave-wide direct load fills 1 KiB (8 rows) of a stage; waves take
    // the 8-row groups round-robin (the B slab may end part way round)
    static constexpr int kLoadsA = BM / 8 / kWaves;
    static constexpr int kLoadsB = (BN / 8 + kWaves - 1) / kWaves;
    static constexpr int kLoadsBMin = BN / 8 / kWaves;  // loads of the wave with the fewest
    static constexpr int kStageA = BM * 128;
    static constexpr int kStageB = BN * 128;
    // every wave's columns lie in one 128-column scale block
    static constexpr bool kOneScaleB = BN % 128 == 0 && 128 % WN == 0;
    // LDS row pitch of the bf16 output tile: a power of two of 16-byte
    // chunks, at least 16, so the chunk swizzle c ^ (row & 15) stays in the row
    static constexpr int kPitchChunks = BN <= 128 ? 16 : 32;
    // the bf16 output tile reuses the stage memory on its way out
    static constexpr int kSmem = (2 * (kStageA + kStageB) > BM * kPitchChunks * 16)
                                     ? 2 * (kStageA + kStageB)
                                     : BM * kPitchChunks * 16;
    static_assert(WM % 16 == 0 && WN % 16 == 0, "wave tile must be a multiple of 16x16");
    static_assert(BM % (8 * kWaves) == 0 && BN % 8 == 0, "slabs are staged 8 rows at a time");
    static_assert(BN <= 256, "output tile pitch");
    static_assert(BM % 64 == 0 && kWaves % (BM / 64) == 0, "waves stage the A scales 64 rows each");
};

// Logical tile of workgroup `b` among `tiles`: XCD x (= b % 8) receives the
// contiguous range [x*per, (x+1)*per); -1 for the padding slots.
__device__ __forceinline__ int xcd_tile(int b, int tiles) {
    const int per = (tiles + kNumXcds - 1) / kNumXcds;
    const int t = (b % kNumXcds) * per + b / kNumXcds;
    return t < tiles ? t : -1;
}

// Where one output tile lives.  Every field is wave-uniform.
struct TileInfo {
    int g;              // group (0 for dense)
    int m0, n0;         // first row within the group's row space, first column
    int valid;          // tile rows [0, valid) exist and may be routed
    int64_t arow0;      // A / sa / D row of tile row 0
    uint64_t ok0, ok1;  // contiguous form: routed-row masks, tile rows 0-63 / 64-127
};

// Contiguous form: the largest valid group id below `below` among the ids of a
// 128-row block (lane l has those of rows l and 64 + l) and the masks of the rows
// carrying it; false when there is none.
__device__ __forceinline__ bool largest_group(int id0, int id1, int64_t G, int below, TileInfo& ti) {
    auto usable = [&](int id) { return id >= 0 && id < G && id < below; };
    const int largest = max(usable(id0) ? id0 : -1, usable(id1) ? id1 : -1);
    const int gid = (int)wave_max((uint32_t)(largest + 1)) - 1;
    if (gid < 0) return false;
    ti.g = gid;
    ti.ok0 = __ballot(id0 == gid);
    ti.ok1 = __ballot(id1 == gid);
    return true;
}

// The same of the block at ti.m0.  Every wave computes this from the layout itself.
__device__ __forceinline__ bool block_group(const int32_t* __restrict__ layout, int64_t G, int below,
                                            int lane, TileInfo& ti) {
    return largest_group(layout[ti.m0 + lane], layout[ti.m0 + 64 + lane], G, below, ti);
}

// An output tile passes through LDS in bf16 and is written back
// in full 16-byte chunks, consecutive lanes on consecutive chunks of a row.  In
// LDS (row pitch kPitchChunks chunks), 16-byte chunk c of row r sits at
// c ^ (r & 15): the 16 rows a fragment store touches land in distinct banks.
//
// Four columns of a row, rounded to bf16 (v_cvt_pk_bf16_f32: nearest even).
template <class T>
__device__ __forceinline__ void stage_bf16(uint8_t* sD, int row, int col, const v4f& v) {
    const v2f lo = {v[0], v[1]};
    const v2f hi = {v[2], v[3]};
    v2u packed;
    packed[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, v2bf));
    packed[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, v2bf));
    *reinterpret_cast<v2u*>(sD + row * (T::kPitchChunks * 16) + (((col >> 3) ^ (row & 15)) << 4) +
                            ((col >> 2) & 1) * 8) = packed;
}

// The staged tile to memory; kRouted: only the rows of ok0 and ok1.
template <class T, bool kRouted>
__device__ __forceinline__ void store_staged(const uint8_t* sD, int tid, const TileInfo& ti, uint16_t* __restrict__ D,
                                             int64_t N) {
    constexpr int kRowBytes = T::kPitchChunks * 16;
    constexpr int kChunks = T::BN / 8;  // 16-byte chunks of an output row
    static_assert((T::BM * kChunks) % T::kThreads == 0, "whole passes over the output tile");
    // fully unrolled (the accumulators are dead by now): every pass's LDS
    // read can be in flight before the first store waits for its data
#pragma unroll
    for (int q = tid; q < T::BM * kChunks; q += T::kThreads) {
        const int row = q / kChunks, c = q % kChunks;
        const int64_t col = ti.n0 + c * 8;
        bool ok = row < ti.valid && col < N;
        if (kRouted) ok = ok && (((row < 64 ? ti.ok0 : ti.ok1) >> (row & 63)) & 1);
        const v4u v = *reinterpret_cast<const v4u*>(sD + row * kRowBytes + ((c ^ (row & 15)) << 4));
        // D is written once and not read back here: non-temporal stores keep
        // it from evicting operand slabs that later tiles still read
        if (ok) __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(D + (ti.arow0 + row) * N + col));
    }
}

// Compute units of the current device, cached per device.  Host threads may
// launch concurrently: each slot only ever receives its device's one value,
// so relaxed atomics suffice.
inline int device_cus() {
    static std::atomic<int> cached[64] = {};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) dev = 0;
    const bool slot = dev >= 0 && dev < 64;
    if (slot) {
        const int c = cached[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
        n = 256;
    if (slot) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace dg
