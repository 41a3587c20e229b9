// Which form a dispatch call takes.  Plain arithmetic, so that a host compiler
// takes it too.
#pragma once

#include <cstdint>

namespace dg {

constexpr int kZeroRows = 16;  // bf16: rows that one workgroup sets to zero where they are padding

// Workgroups of the copies that sort for themselves: a token's parts in bf16
// (rows of 8 columns, and those that clear padding) and in codes of 128 columns,
// a token each in int8.
inline int64_t small_grid_bf16(int64_t T, int64_t H, int64_t M) {
    return T * ((H / 8 + 255) / 256) + (M + kZeroRows - 1) / kZeroRows;
}
inline int64_t small_grid_fp8(int64_t T, int64_t H) { return T * ((H / 128 + 31) / 32); }

// Whether every workgroup of the copies sorts for itself, instead of copying
// behind a sort of its own launches.  That saves two launches, and costs each of
// the `grid` workgroups a count of all pairs in LDS, whose additions to one
// expert follow each other, and a walk over the experts: grid * (P (1 + 16 / E) +
// E / 4) steps, of which about 16 million take as long as the launches.  In us,
// by themselves and behind a sort:
//   FP8   512 tokens to 8 of 256, 7168:    11.5 and 17.7     (4.9 million)
//   FP8  4096 tokens to 1 of 256, 7168:    32.2 and 25.1    (36)
//   FP8  4096 tokens to 1 of 2, 7168:      107  and 24.0    (302)
//   bf16  333 tokens to 5 of 31, 1024:      8.0 and 12.0     (1.7)
//   bf16  128 tokens to 8 of 1024, 1024:   39.7 and 51.9    (11)
//   bf16 2048 tokens to 2 of 8, 7168:      49.2 and 25.3   (100)
//   bf16 4096 tokens to 1 of 4096, 256:    563  and 76.8   (191)
//   int8 1024 tokens to 1 of 8, 7168:       9.0 and 10.9     (3.1)
// Over 645 sizes up to 4096 pairs the form that is taken is 0.8% slower than the
// faster one on average; 42% if pairs alone decide.  P is at most kSmallPairs,
// which the steps' count is measured for.
constexpr int64_t kSmallPairs = 4096;
constexpr int64_t kSmallSteps = 16000000;
inline bool sorts_for_itself(int64_t P, int64_t E, int64_t grid) {
    return P > 0 && P <= kSmallPairs && grid <= kSmallSteps / (P + 16 * P / E + E / 4);
}

}  // namespace dg
