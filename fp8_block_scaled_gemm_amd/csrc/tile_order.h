// The order of a contiguous-grouped product's tiles.  Plain arithmetic, so that
// a host compiler takes it too.
//
// Workgroup b runs on XCD b % 8.  Each XCD takes a run of blocks, rasterized like
// the dense form, so that few XCDs read one group's weights.  A buffer of the
// most rows that any choice of experts needs holds them at its beginning, and a
// run of the whole buffer's blocks would leave them to one of the eight; so the
// runs cover the part in use, as far as 16 evenly spread blocks show it.  Behind
// it tiles go in plain order, the columns of a block first, which spreads what is
// left over all XCDs.  So do wide buffers of many tiles, where a share of every
// block's columns for each XCD is the better one.
// In us, runs of the whole buffer / plain order / this one:
//   8 groups of 4096 rows, 2112 x 7168: 541 / 710 / 545; an eighth in use 454 / 160 / 124
//   64 groups of 512, 512 x 7168:       144 / 215 / 142
//   32 groups of 1024, 768 x 2048:     61.8 / 97.5 / 62.7
//   128 groups of 128, 1024 x 4096:     160 / 170 / 158
//   8 groups of 4096, 4096 x 1024:      210 / 180 / 183 (wide)
//   8 groups of 4096, 4096 x 7168:     1013 / 988 / 997 (wide); an eighth in use 779 / 147 / 145
//   8 groups of 512, 7168 x 512:       33.4 / 37.0 / 33.8 (896 tiles)
#pragma once

#include <cstdint>

namespace dg {

constexpr int kNumXcds = 8;
constexpr int kLooks = 16;  // blocks looked at
constexpr int kWideBlocks = 16, kWideTiles = 2048;

struct Place {
    int m, n;  // block of 128 rows, column tile
};

__device__ __forceinline__ bool wide_buffer(int m_blocks, int n_blocks) {
    return n_blocks >= kWideBlocks && m_blocks * n_blocks >= kWideTiles;
}

// The block that look l in [0, kLooks) looks at; -1: none.
__device__ __forceinline__ int look_at(int l, int m_blocks) { return (int)((int64_t)(l + 1) * m_blocks / kLooks) - 1; }

// The blocks in runs, where look `upto` - 1 is the last one that found a group:
// whole ones for each XCD, so that plain order goes on where the runs end.
__device__ __forceinline__ int run_blocks(int upto, int m_blocks) {
    return (int)((int64_t)upto * m_blocks / kLooks) / kNumXcds * kNumXcds;
}

__device__ __forceinline__ Place plain_place(int b, int n_blocks) { return {b / n_blocks, b % n_blocks}; }

// For b below run * n_blocks: groups of group_m blocks, blocks first within one.
__device__ __forceinline__ Place run_place(int b, int run, int n_blocks, int group_m) {
    const int tile = b % kNumXcds * (run / kNumXcds * n_blocks) + b / kNumXcds;
    const int span = group_m * n_blocks;
    const int first = tile / span * group_m, within = tile % span;
    const int rows = run - first < group_m ? run - first : group_m;
    return {first + within % rows, within / rows};
}

}  // namespace dg
