"""Dispatch calls of few pairs whose grids pass 2^22 workgroups, by the rows of
their buffers or by a token's width: the layout's shares count in 32 bits."""
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [2 ** 26, 2 ** 27, 2 ** 28 - 1024])
def test_one_token_into_a_buffer_of_many_rows(M):
    x = torch.arange(1, 9, dtype=torch.bfloat16, device="cuda").view(1, 8)
    ids = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    out = torch.full((M, 8), 5.0, dtype=torch.bfloat16, device="cuda")
    layout = torch.full((M,), 7, dtype=torch.int32, device="cuda")
    got, rows, _, offsets = dg.dg_moe_dispatch(x, ids, 1, out, None, layout)
    assert rows.tolist() == [[0]] and offsets.tolist() == [0, 128]
    assert int(layout[0]) == 0 and int(layout[1:].max()) == -1 and int(layout[1:].min()) == -1
    assert torch.equal(got[:1], x)
    assert not bool(got[1:].view(torch.int16).any())


@pytest.mark.parametrize("kind,H", [("bf16", 2 ** 21), ("fp8", 2 ** 22), ("e8m0", 2 ** 22)])
def test_wide_tokens(kind, H):
    T = 4096
    value = (torch.arange(T, device="cuda") % 241 + 1).to(torch.bfloat16)
    x = value.view(T, 1).repeat(1, H)
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    call = {"bf16": dg.dg_moe_dispatch, "fp8": dg.dg_moe_dispatch_fp8, "e8m0": dg.dg_moe_dispatch_fp8_e8m0}[kind]
    got = call(x, ids, 1)
    rows, layout, offsets = got[-3:]
    assert torch.equal(rows.flatten(), torch.arange(T, dtype=torch.int32, device="cuda")) and offsets.tolist() == [0, T]
    assert layout.numel() == T and int(layout.abs().max()) == 0
    del x
    if kind == "bf16":
        for r in range(0, T, 512):
            assert bool((got[0][r:r + 512] == value[r:r + 512, None]).all())
        return
    small = value.view(T, 1).repeat(1, 128).float()
    q, s = (dg.dg_quantize_fp8_per_token if kind == "fp8" else dg.dg_quantize_fp8_per_token_e8m0)(small)
    for r in range(0, T, 512):
        assert bool((got[0][r:r + 512] == q[r:r + 512, :1]).all())
        assert bool((got[1][r:r + 512] == s[r:r + 512, :1]).all())
