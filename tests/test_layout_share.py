"""The shares of a layout's rows (csrc/layout_share.h) on the host: whatever the
number of workgroups, every row is written once and nothing else is, and no
32-bit product overflows on the way."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "layout_share.h"

// workgroups, their waves, rows M, and each expert's pairs: as a launch of so many workgroups writes its layout
int main(int argc, char** argv) {
    const unsigned workgroups = strtoul(argv[1], nullptr, 0);
    const int each = atoi(argv[2]);
    const int64_t M = atoll(argv[3]);
    std::vector<int> size, offsets{0};
    for (int i = 4; i < argc; ++i) {
        size.push_back(atoi(argv[i]));
        offsets.push_back(offsets.back() + (size.back() + 127) / 128 * 128);
    }
    const int E = (int)size.size();
    std::vector<uint8_t> times(M, 0);
    int64_t outside = 0;
    auto touch = [&](int64_t at) {
        if (at < 0 || at >= M) ++outside;
        else if (times[at] < 255) ++times[at];
    };
    const int waves = dg::layout_waves(workgroups, each);
    if (waves <= E || waves > (int64_t)workgroups * each) return 2;
    for (int wave = 0; wave < waves; ++wave) {
        const dg::BlockShare s = dg::block_share(wave, waves, E);
        if (s.expert < 0 || s.expert >= E || s.begin < 0 || s.step < 1) return 3;
        dg::each_block(size[s.expert], s.begin, s.step, [&](int r) {
            for (int i = 0; i < 128; ++i) touch((int64_t)offsets[s.expert] + r + i);
        });
        for (int lane = 0; lane < 64; ++lane)
            dg::each_rest(offsets[E], M, wave, waves, lane, [&](int64_t r) {
                for (int i = 0; i < 4; ++i) touch(r + i);
            });
    }
    int64_t wrong = 0;
    for (uint8_t t : times) wrong += t != 1;
    printf("%lld outside, %lld not once\n", (long long)outside, (long long)wrong);
    return outside == 0 && wrong == 0 ? 0 : 1;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("layout_share")
    (d / "share.cpp").write_text(PROGRAM)
    # a signed overflow ends the program instead of wrapping
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
                    "-D__device__=", "-D__forceinline__=inline", f"-I{ROOT}/fp8_block_scaled_gemm_amd/csrc",
                    str(d / "share.cpp"), "-o", str(d / "share")], check=True)
    return str(d / "share")


@pytest.mark.parametrize("workgroups,each,M,sizes", [
    (1, 16, 512, [130, 0, 1]), (3, 4, 1024, [200, 127, 129, 0, 0]), (8, 4, 4224, [4096]),
    (257, 4, 70000 // 128 * 128, [1, 300, 5, 0, 1000]),
    (1 << 22, 4, 1 << 12, [1]), ((1 << 22) + 1, 4, 1 << 20, [4096]),        # 2^24 waves for one expert
    (1 << 23, 4, 1 << 13, [4096, 1]), (3 << 22, 4, 1 << 13, [2000, 0, 2096]),  # for two and three
    ((1 << 24) - 1, 4, 1 << 26, [3000]),                                    # as many as a grid holds
])
def test_every_row_is_written_once(program, workgroups, each, M, sizes):
    got = subprocess.run([program, str(workgroups), str(each), str(M), *map(str, sizes)], capture_output=True, text=True,
                         timeout=120)
    assert got.returncode == 0, got.stdout + got.stderr
