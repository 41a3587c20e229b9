// How the waves of a launch share out the rows of a layout.  Plain arithmetic,
// so that a host compiler takes it too.
#pragma once

#include <cstdint>

namespace dg {

// The waves that take part among those of `workgroups` of `each`: the first 2^16
// at most.  A grid has up to 2^26, whose shares in rows pass 32 bits; of so many
// as take part, wave and step times a share's 256 rows stay below 2^24.
constexpr int kLayoutWaves = 1 << 16;
__device__ __forceinline__ int layout_waves(unsigned workgroups, int each) {
    return workgroups < (unsigned)(kLayoutWaves / each) ? (int)workgroups * each : kLayoutWaves;
}

// Where there are more waves than experts: the expert whose 128-row blocks a
// wave writes, and which of them, every step-th from begin on.
struct BlockShare {
    int expert, begin, step;
};
__device__ __forceinline__ BlockShare block_share(int wave, int waves, int E) {
    return {wave % E, wave / E, (waves - 1 - wave % E) / E + 1};
}

// write(r) for the first row of each such block of an expert of n rows, n at most
// 2^30 and begin and step below kLayoutWaves.
template <class Write>
__device__ __forceinline__ void each_block(int n, int begin, int step, Write write) {
    for (int r = begin * 128; r < n; r += step * 128) write(r);
}

// write(r) for the first of each four rows from `first` on that a lane writes.
template <class Write>
__device__ __forceinline__ void each_rest(int64_t first, int64_t M, int wave, int waves, int lane, Write write) {
    for (int64_t r = first + ((int64_t)wave * 64 + lane) * 4; r < M; r += (int64_t)waves * 256) write(r);
}

}  // namespace dg
