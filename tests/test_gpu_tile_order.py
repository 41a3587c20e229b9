"""Contiguous-grouped products whose buffers are used in part, at sizes that
take either order of the tiles (tests/test_tile_order.py): every row as in a
buffer of its group alone, every row of padding as it was."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg

pytestmark = pytest.mark.gpu


def codes(rng, *n):
    q = rng.integers(0, 256, n, dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] ^= 1
    return torch.from_numpy(q).cuda()


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("sizes,behind,N", [
    ([300, 0, 128, 77], 0, 264), ([300, 0, 128, 77], 5, 264), ([128] * 40, 260, 520), ([700, 1, 900], 30, 2112),
    ([129] * 33, 0, 1544), ([2000, 1500, 10], 100, 4104), ([128] * 130, 3, 4104), ([5], 15, 8), ([640, 640], 1, 1032),
])
def test_rows_as_in_a_buffer_of_their_own(kind, sizes, behind, N):
    rng = np.random.default_rng(len(sizes) + N)
    G, K = len(sizes), 256
    layout = np.concatenate([np.where(np.arange(-(-s // 128) * 128) < s, g, -1) for g, s in enumerate(sizes)]
                            + [np.full(128 * behind, -1)]).astype(np.int32)
    M = layout.size
    A, B = codes(rng, M, K), codes(rng, G, N, K)
    if kind == "fp32":
        call = dg.dg_fp8_gemm_grouped_contiguous
        sa = torch.from_numpy(rng.random((M, 2), dtype=np.float32) + 0.5).cuda()
        sb = torch.from_numpy(rng.random((G, (N + 127) // 128, 2), dtype=np.float32) + 0.5).cuda()
    else:
        call = dg.dg_fp8_gemm_grouped_contiguous_e8m0
        sa = torch.from_numpy(rng.integers(124, 130, (M, 4), dtype=np.uint8)).cuda()
        sb = torch.from_numpy(rng.integers(124, 130, (G, (N + 127) // 128, 4), dtype=np.uint8)).cuda()
    lay = torch.from_numpy(layout).cuda()
    D = torch.full((M, N), 77, dtype=torch.int16, device="cuda")
    call(A, sa, B, sb, D, lay)
    assert bool((D[lay < 0] == 77).all())
    first = 0
    for g, s in enumerate(sizes):
        n = -(-s // 128) * 128
        if n:
            one = torch.empty(n, N, dtype=torch.int16, device="cuda")
            call(A[first:first + n], sa[first:first + n], B[g:g + 1], sb[g:g + 1].clone(), one,
                 torch.zeros(n, dtype=torch.int32, device="cuda"))
            assert torch.equal(D[first:first + s], one[:s])
        first += n
    # rows in use behind a gap that the looks miss
    late = torch.full_like(lay, -1)
    late[M - 128:] = G - 1
    D.fill_(77)
    call(A, sa, B, sb, D, late)
    one = torch.empty(128, N, dtype=torch.int16, device="cuda")
    call(A[M - 128:], sa[M - 128:], B[G - 1:], sb[G - 1:].clone(), one, torch.zeros(128, dtype=torch.int32, device="cuda"))
    assert torch.equal(D[M - 128:], one) and bool((D[:M - 128] == 77).all())
