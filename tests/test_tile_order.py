"""The order of a contiguous-grouped product's tiles (csrc/tile_order.h) on the
host: every tile has one workgroup, few XCDs read a group's weights, and the
part of a buffer that is in use is shared out over all of them."""
import subprocess

import pytest

from tests.test_layout_share import ROOT

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "tile_order.h"

// m_blocks, n_blocks, used blocks: the tile of each workgroup
int main(int, char** argv) {
    const int m_blocks = atoi(argv[1]), n_blocks = atoi(argv[2]), used = atoi(argv[3]);
    int upto = 0;
    for (int l = 0; l < dg::kLooks; ++l) {
        const int at = dg::look_at(l, m_blocks);
        if (at >= m_blocks) return 2;
        if (at >= 0 && at < used) upto = l + 1;
    }
    const int run = dg::wide_buffer(m_blocks, n_blocks) ? 0 : dg::run_blocks(upto, m_blocks);
    for (int b = 0; b < m_blocks * n_blocks; ++b) {
        const dg::Place p = b < run * n_blocks ? dg::run_place(b, run, n_blocks, 8) : dg::plain_place(b, n_blocks);
        printf("%d %d\n", p.m, p.n);
    }
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    d = tmp_path_factory.mktemp("tile_order")
    (d / "order.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
                    "-D__device__=", "-D__forceinline__=inline", f"-I{ROOT}/fp8_block_scaled_gemm_amd/csrc",
                    str(d / "order.cpp"), "-o", str(d / "order")], check=True)

    def of(m_blocks, n_blocks, used):
        out = subprocess.run([str(d / "order"), str(m_blocks), str(n_blocks), str(used)], capture_output=True, text=True,
                             check=True).stdout.split()
        return list(zip(map(int, out[::2]), map(int, out[1::2])))
    return of


@pytest.mark.parametrize("m_blocks,n_blocks", [(1, 1), (2, 3), (7, 9), (8, 1), (9, 2), (33, 9), (64, 3), (65, 28), (73, 28),
                                               (128, 16), (263, 8), (263, 16), (1000, 1)])
def test_every_tile_has_one_workgroup(order, m_blocks, n_blocks):
    for used in {0, 1, m_blocks // 8, m_blocks // 2, m_blocks - 1, m_blocks}:
        got = order(m_blocks, n_blocks, used)
        assert sorted(got) == [(m, n) for m in range(m_blocks) for n in range(n_blocks)]


@pytest.mark.parametrize("groups,blocks,n_blocks", [(64, 4, 1), (64, 4, 2), (64, 4, 3), (64, 4, 6), (32, 8, 9), (32, 8, 8)])
def test_few_xcds_read_a_groups_weights(order, groups, blocks, n_blocks):
    readers = [set() for _ in range(groups)]
    for b, (m, _) in enumerate(order(groups * blocks, n_blocks, groups * blocks)):
        readers[m // blocks].add(b % 8)
    assert sum(map(len, readers)) <= groups + 8  # one each, two where a run ends


@pytest.mark.parametrize("m_blocks,n_blocks,used", [(263, 9, 33), (263, 9, 130), (510, 8, 400), (256, 2, 128), (64, 16, 9),
                                                    (263, 16, 33), (40, 3, 40), (510, 6, 300)])
def test_rows_in_use_are_shared_out_over_all_xcds(order, m_blocks, n_blocks, used):
    share = [0] * 8
    for b, (m, _) in enumerate(order(m_blocks, n_blocks, used)):
        share[b % 8] += m < used
    assert max(share) - min(share) <= n_blocks
