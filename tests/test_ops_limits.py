"""CPU tests of the sizes at the ends of the ranges of include/dg_ops.h: no
rows, and launches past what a grid can hold."""
import ctypes
import os

import pytest

import fp8_block_scaled_gemm_amd as dg

DG_OK = 0


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.library_path()):
        from fp8_block_scaled_gemm_amd import build
        build.build()
    return dg.load_library()


@pytest.mark.parametrize("N,K,L,R", [(128, 256, 4, 16), (8, 128, 1, 8), (65536, 65536, 65536, 128)])
def test_lora_workspace_of_no_rows(lib, N, K, L, R):
    n = ctypes.c_int64(-1)
    assert lib.dg_fp8_gemm_nt_lora_workspace(0, N, K, L, R, ctypes.byref(n)) == DG_OK
    assert n.value == 0


def test_moe_workspace_of_no_tokens(lib):
    n = ctypes.c_int64(-1)
    assert lib.dg_moe_mlp_fp8_workspace(0, 2, 8, 256, 128, ctypes.byref(n)) == DG_OK
    assert n.value >= 0


# A grid dimension holds 2^32 - 1 work-items; past that a launch runs a part of
# its workgroups and reports nothing.
FAKE, DG_ERR_SHAPE = 0x10000, 2  # FAKE: never dereferenced, the checks reject first


@pytest.mark.parametrize("name", ["dg_fp8_gemm_nt_lora", "dg_fp8_gemm_nt_lora_e8m0"])
@pytest.mark.parametrize("M,N,R", [((1 << 31) - 1, 1024, 8),   # the dense tiles
                                   (1 << 30, 8, 64), (1 << 29, 8, 16), (1 << 28, 8, 128)])  # the first product
def test_lora_refuses_more_work_items_than_a_grid_holds(lib, name, M, N, R):
    n = ctypes.c_int64(-1)
    assert lib.dg_fp8_gemm_nt_lora_workspace(M, N, 128, 2, R, ctypes.byref(n)) == DG_ERR_SHAPE
    assert getattr(lib, name)(*[FAKE] * 10, M, N, 128, 2, R, FAKE, 1 << 62, None) == DG_ERR_SHAPE


def test_lora_takes_sizes_up_to_a_full_grid(lib):
    n = ctypes.c_int64(-1)
    for M, N, R in ((1 << 27, 8, 16), ((1 << 28) - 32, 8, 64), (1 << 25, 8192, 16)):
        assert lib.dg_fp8_gemm_nt_lora_workspace(M, N, 128, 2, R, ctypes.byref(n)) == DG_OK and n.value >= M * R * 4


def test_products_and_quantizers_refuse_more_work_items_than_a_grid_holds(lib):
    for name in ("dg_fp8_gemm_grouped_masked", "dg_fp8_gemm_grouped_masked_e8m0"):
        # 2^23 groups of one tile of 512 work-items
        assert getattr(lib, name)(*[FAKE] * 6, 1 << 23, 1, 8, 128, None) == DG_ERR_SHAPE
    # 2^24 workgroups of 256
    assert lib.dg_quantize_fp8_per_token(FAKE, 1 << 22, 1 << 14, FAKE, FAKE, None) == DG_ERR_SHAPE
    assert lib.dg_quantize_fp8_per_token_bf16(FAKE, 1 << 22, 1 << 14, FAKE, FAKE, None) == DG_ERR_SHAPE
    assert lib.dg_quantize_fp8_per_block(FAKE, 1, 1 << 31, FAKE, FAKE, None) == DG_ERR_SHAPE
