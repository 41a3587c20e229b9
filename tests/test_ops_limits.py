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
