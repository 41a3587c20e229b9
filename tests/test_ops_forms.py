"""Which form the adapters' call takes at the sizes of its GPU tests, so that a
change of the rule cannot leave a test of one form running the other.  The
few-row form keeps fp32 sums [shares][M][N] behind the vectors in its
workspace; the dense tiles keep the vectors [parts][M][R] alone."""
import pytest

import fp8_block_scaled_gemm_amd as dg
from tests.test_ops_limits import lib  # noqa: F401  (fixture: builds what is missing)

DENSE = [  # M, N, K, R, L
    (1540, 328, 256, 72, 5),                                    # every tile shape
    (1540, 136, 256, 16, 4), (1540, 264, 256, 24, 3),           # infinities; graph and stream
    (33, 4096, 128, 128, 1), (50, 3000, 128, 128, 4), (160, 1032, 256, 128, 3), (257, 1032, 384, 72, 2),
    (1540, 136, 256, 40, 64), (1552, 264, 640, 24, 6), (1537, 8, 128, 64, 600), (1600, 256, 1152, 16, 2),
    (1540, 136, 256, 24, 6), (1540, 136, 256, 72, 6), (1540, 136, 256, 104, 6),  # values that are not finite
    (1540, 2048, 2048, 128, 10000), (1540, 8, 32768, 72, 1024),  # adapters past 4 GiB
    (8189, 40, 128, 8, 1024), (8193, 40, 128, 8, 5),
]
FEW = [(20, 136, 256, 24, 6), (20, 136, 256, 104, 6), (300, 136, 256, 24, 6), (3, 2048, 2048, 128, 10000),
       (64, 256, 512, 40, 64), (515, 72, 384, 24, 16)]


def up(n):
    return (n + 255) // 256 * 256


def vectors_only(M, N, K, R, L):
    return dg.dg_fp8_gemm_nt_lora_workspace(M, N, K, L, R) in [up(parts * M * R * 4) for parts in (1, 2, 3, 4)]


@pytest.mark.parametrize("sizes", DENSE)
def test_sizes_that_take_dense_tiles(lib, sizes):  # noqa: F811
    assert vectors_only(*sizes)


@pytest.mark.parametrize("sizes", FEW)
def test_sizes_that_take_the_few_row_form(lib, sizes):  # noqa: F811
    assert not vectors_only(*sizes)
