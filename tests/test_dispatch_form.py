"""Which form a dispatch call takes (csrc/dispatch_form.h), on the host: copies
that sort for themselves only where that is the faster form, and never in a
grid so large that it could not be launched."""
import subprocess

import pytest

from tests import experts_ref as ref
from tests.test_layout_share import ROOT

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "dispatch_form.h"

// held T k E H M ...: 1 where the copies sort for themselves
int main(int argc, char** argv) {
    for (int i = 1; i + 5 < argc; i += 6) {
        const int64_t T = atoll(argv[i + 1]), k = atoll(argv[i + 2]), E = atoll(argv[i + 3]), H = atoll(argv[i + 4]);
        const int64_t grid = !strcmp(argv[i], "bf16")   ? dg::small_grid_bf16(T, H, atoll(argv[i + 5]))
                             : !strcmp(argv[i], "int8") ? T
                                                        : dg::small_grid_fp8(T, H);
        printf("%d %lld\n", (int)dg::sorts_for_itself(T * k, E, grid), (long long)grid);
    }
}
"""


@pytest.fixture(scope="module")
def form(tmp_path_factory):
    d = tmp_path_factory.mktemp("dispatch_form")
    (d / "form.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
                    f"-I{ROOT}/fp8_block_scaled_gemm_amd/csrc", str(d / "form.cpp"), "-o", str(d / "form")], check=True)

    def of(*sizes):
        args = [str(v) for held, T, k, E, H, *M in sizes for v in (held, T, k, E, H, M[0] if M else ref.sort_rows(T, k, E))]
        got = subprocess.run([str(d / "form"), *args], capture_output=True, text=True, check=True).stdout.split()
        return [(int(a), int(b)) for a, b in zip(got[::2], got[1::2])]
    return of


@pytest.mark.parametrize("sizes,us", [  # in us: by themselves and behind a sort, where they differ by a tenth or more
    (("fp8", 1, 8, 256, 7168), (6.4, 9.6)), (("fp8", 512, 8, 256, 7168), (11.5, 17.7)), (("fp8", 333, 5, 31, 1024), (6.0, 11.1)),
    (("fp8", 512, 8, 4096, 256), (25.3, 39.0)), (("fp8", 1024, 1, 1, 7168), (18.4, 11.2)), (("fp8", 4096, 1, 1, 7168), (180, 24.4)),
    (("fp8", 4096, 1, 2, 256), (54.4, 10.5)), (("fp8", 4096, 1, 256, 7168), (32.2, 25.1)), (("fp8", 2048, 2, 8, 7168), (28.8, 19.5)),
    (("fp8", 4096, 1, 4096, 7168), (131, 50.8)), (("bf16", 16, 8, 256, 7168), (33.1, 37.3)), (("bf16", 333, 5, 31, 1024), (8.0, 12.0)),
    (("bf16", 128, 8, 1024, 1024), (39.7, 51.9)), (("bf16", 512, 1, 1, 16384), (19.7, 10.0)), (("bf16", 2048, 2, 8, 7168), (49.2, 25.3)),
    (("bf16", 4096, 1, 1, 7168), (349, 26.2)), (("bf16", 4096, 1, 4096, 256), (563, 76.8)), (("bf16", 512, 8, 4096, 256), (541, 76.3)),
    (("int8", 1, 8, 256, 7168), (9.0, 11.0)), (("int8", 1024, 1, 8, 7168), (9.0, 10.9)), (("int8", 512, 8, 64, 7168), (12.7, 16.9)),
    (("int8", 4096, 1, 1, 7168), (93.2, 27.3)), (("int8", 2048, 1, 1, 1024), (29.2, 12.2)), (("int8", 4096, 1, 4096, 256), (69.2, 40.4)),
])
def test_the_faster_form_is_taken(form, sizes, us):
    assert form(sizes)[0][0] == (us[0] < us[1])


def test_more_pairs_are_sorted_first(form):
    # 4096 and 4097 pairs in as many workgroups as tokens; 4096 of one choice: 15.8 us by themselves, 12.1 behind a sort
    assert [a for a, _ in form(("fp8", 512, 8, 256, 128), ("int8", 64, 64, 256, 128), ("fp8", 4096, 1, 256, 128),
                               ("int8", 241, 17, 256, 128), ("fp8", 0, 8, 256, 128))] == [1, 1, 0, 0, 0]


def test_no_grid_of_many_workgroups_sorts_for_itself(form):
    wide = [(held, T, k, E, H) for held in ("bf16", "fp8") for T, k in ((4096, 1), (512, 8), (1, 1)) for E in (1, 3, 16, 4096)
            for H in (2 ** 21, 2 ** 22, 2 ** 24 - 128)]
    deep = [("bf16", 1, 1, E, 8, M) for E in (1, 2, 10, 64, 4096) for M in (2 ** 24, 2 ** 26, 2 ** 28 - 1024, 2 ** 31 - 128)]
    for taken, grid in form(*wide, *deep):
        assert not taken or grid < 2 ** 22
    assert [a for a, _ in form(*deep)][-1] == 0
