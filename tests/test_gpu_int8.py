"""The int8 products and their quantizer (include/dg_int8.h) on the GPU: the
sum is exact and every later rounding is defined, so results are compared bit
by bit."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import experts_ref as ref
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu

SENTINEL = -1


def bits(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy()


def operands(rng, M, N, K, G=None):
    A = rng.integers(-128, 128, (M, K)).astype(np.int8)
    B = rng.integers(-128, 128, (N, K) if G is None else (G, N, K)).astype(np.int8)
    sa = (rng.random(M).astype(np.float32) + np.float32(0.01)) / 127
    sb = rng.standard_normal(N if G is None else (G, N)).astype(np.float32)
    return A, sa, B, sb


DENSE = [(1, 8, 128), (1, 7168, 2048), (2, 40, 384), (3, 520, 1152), (5, 1032, 256), (7, 24, 5120), (8, 264, 640),
         (9, 264, 640), (15, 136, 256), (16, 72, 1024), (17, 1000, 384), (31, 8, 2176), (33, 328, 512), (64, 2112, 7168),
         (32, 40, 128), (64, 512, 7168), (40, 8, 8320), (255, 1016, 640),
         (100, 264, 256), (127, 56, 128), (129, 520, 384), (256, 256, 128), (257, 264, 256), (300, 4104, 640),
         (512, 8192, 256), (1000, 2064, 384), (2049, 4088, 128), (4096, 2112, 256),
         # 192 and 160 columns behind a round of 256 (256 CUs)
         (4096, 7168, 128), (4090, 6648, 256), (4096, 6656, 128)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense_matches_definition(M, N, K):
    rng = np.random.default_rng(M + N + K)
    A, sa, B, sb = operands(rng, M, N, K)
    D = torch.full((M + 1, N), SENTINEL, dtype=torch.int16, device="cuda")
    assert dg.dg_int8_gemm_nt(to_dev(A), to_dev(sa), to_dev(B), to_dev(sb), D[:M]).data_ptr() == D.data_ptr()
    got = D.cpu().numpy()
    assert (got[M] == SENTINEL).all()
    assert np.array_equal(got[:M], bits(exact_product(A, sa, B, sb)))


def exact_product(A, sa, B, sb):
    """ref.int8_product with the sums by a 64-bit float product: exact below 2^53."""
    sums = torch.matmul(torch.from_numpy(A).double().cuda(), torch.from_numpy(B).double().cuda().T).cpu().numpy()
    return (sa[:, None] * sb) * sums.astype(np.float32)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("a,b", [(-128, -128), (127, 127), (-128, 127)])
def test_the_longest_sums_do_not_wrap(a, b, M):
    K, N = 2 ** 17 - 128, 8
    A = torch.full((M, K), a, dtype=torch.int8, device="cuda")
    B = torch.full((N, K), b, dtype=torch.int8, device="cuda")
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(max(M, N), device="cuda")
    dg.dg_int8_gemm_nt(A, one[:M].clone(), B, one[:N].clone(), D)
    want = torch.tensor(float(a * b * K), dtype=torch.float32).to(torch.bfloat16)
    assert bool((D.cpu() == want).all())


@pytest.mark.parametrize("M", [1, 20, 200, 600])
def test_scales_that_are_not_finite_stay_in_their_rows_and_columns(M):
    rng = np.random.default_rng(M)
    A, sa, B, sb = operands(rng, M, 264, 256)
    A[0] = 0
    sa[M // 2] = np.nan
    sb[5] = np.inf
    D = torch.empty(M, 264, dtype=torch.bfloat16, device="cuda")
    dg.dg_int8_gemm_nt(to_dev(A), to_dev(sa), to_dev(B), to_dev(sb), D)
    got = D.float().cpu().numpy()
    assert np.isnan(got[M // 2]).all()
    rest = np.arange(M) != M // 2
    assert np.isnan(got[0, 5]) or M // 2 == 0  # 0 times infinity
    assert np.isfinite(np.delete(got[rest], 5, axis=1)).all() and not np.isfinite(got[rest][:, 5]).any()


GROUPED = [(3, 264, 384, [100, 0, 200]), (1, 8, 128, [1]), (5, 520, 256, [128, 1, 127, 0, 130]), (8, 4096, 256, [3] * 8),
           (16, 1032, 640, [5, 0, 300, 17, 128, 64, 0, 0, 90, 33, 12, 1, 2, 16, 31, 257]), (2, 2048, 2048, [700, 900]),
           # left-over tiles as they are, and behind a whole round in halves and in quarters (256 CUs)
           (2, 2048, 256, [1300, 1250]), (3, 2056, 128, [2000, 1500, 1700]), (2, 2048, 128, [2500, 2400]),
           # at most 32 rows a block, and one more
           (4, 264, 128, [32, 1, 0, 7]), (3, 520, 7168, [32, 31, 5]), (3, 1288, 640, [2, 33, 1]), (9, 1024, 384, [9] * 9)]


def grouped_case(G, N, K, counts, seed):
    rng = np.random.default_rng(seed)
    layout = []
    for g, n in enumerate(counts):
        layout += [g] * n + [-1] * (-n % 128)
    layout += [-1] * 128
    layout = np.array(layout, np.int32)
    return (*operands(rng, layout.size, N, K, G), layout)


def check_grouped(D, A, sa, B, sb, layout):
    got = D.cpu().numpy()
    G = B.shape[0]
    for g in range(G):
        r = np.nonzero(layout == g)[0]
        if r.size:
            assert np.array_equal(got[r], bits(exact_product(A[r], sa[r], B[g], sb[g]))), g
    assert (got[(layout < 0) | (layout >= G)] == SENTINEL).all()


@pytest.mark.parametrize("G,N,K,counts", GROUPED)
def test_grouped_matches_definition(G, N, K, counts):
    A, sa, B, sb, layout = grouped_case(G, N, K, counts, N + K)
    D = torch.full((layout.size, N), SENTINEL, dtype=torch.int16, device="cuda")
    dg.dg_int8_gemm_grouped_contiguous(to_dev(A), to_dev(sa), to_dev(B), to_dev(sb), D, to_dev(layout))
    check_grouped(D, A, sa, B, sb, layout)


@pytest.mark.parametrize("N", [264, 1032])
def test_grouped_blocks_that_mix_ids(N):
    A, sa, B, sb, layout = grouped_case(5, N, 384, [128, 100, 0, 256, 30], 9)
    rng = np.random.default_rng(1)
    layout[128:256] = rng.integers(-3, 8, 128)  # several, and some that are none
    layout[300] = 4
    D = torch.full((layout.size, N), SENTINEL, dtype=torch.int16, device="cuda")
    dg.dg_int8_gemm_grouped_contiguous(to_dev(A), to_dev(sa), to_dev(B), to_dev(sb), D, to_dev(layout))
    check_grouped(D, A, sa, B, sb, layout)


@pytest.mark.parametrize("rows", [32, 33])
def test_grouped_blocks_that_mix_ids_in_their_first_rows(rows):
    A, sa, B, sb, layout = grouped_case(5, 264, 384, [128, 100, 0, 256, 30], 9)
    rng = np.random.default_rng(rows)
    ids = np.full((layout.size // 128, 128), -1, np.int32)
    ids[:4, :rows] = rng.integers(-3, 8, (4, rows))
    ids[2, :rows] = 2 ** 31 - 1
    ids[0, rows - 1] = 4
    layout = ids.reshape(-1)
    D = torch.full((layout.size, 264), SENTINEL, dtype=torch.int16, device="cuda")
    dg.dg_int8_gemm_grouped_contiguous(to_dev(A), to_dev(sa), to_dev(B), to_dev(sb), D, to_dev(layout))
    check_grouped(D, A, sa, B, sb, layout)


def test_grouped_blocks_far_apart_in_a_long_buffer():
    """Few blocks that hold rows, the others empty, over more of them than a workgroup lists at once."""
    rng = np.random.default_rng(3)
    M, N, K, G = 9000 * 128, 264, 128, 3
    layout = np.full(M, -1, np.int32)
    for b in (0, 63, 64, 1000, 4095, 4096, 4097, 8191, 8192, 8999):
        layout[b * 128 + rng.integers(0, 128, 40)] = rng.integers(0, G)
    layout[5000 * 128 + 127], layout[6000 * 128:6001 * 128] = 2, G  # one row alone; ids that are none
    rows = np.nonzero((layout >= 0) & (layout < G))[0]
    A = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda")
    B = torch.randint(-128, 128, (G, N, K), dtype=torch.int8, device="cuda")
    sa, sb = torch.rand(M, device="cuda"), torch.rand(G, N, device="cuda")
    D = torch.full((M, N), SENTINEL, dtype=torch.int16, device="cuda")
    dg.dg_int8_gemm_grouped_contiguous(A, sa, B, sb, D, to_dev(layout))
    at = torch.from_numpy(rows).cuda()
    want = exact_rows(A[at], sa[at], B, sb, torch.from_numpy(layout[rows].astype(np.int64)).cuda())
    assert torch.equal(D[at].view(torch.bfloat16), want)
    D[at] = SENTINEL
    assert bool((D == SENTINEL).all())


def exact_rows(A, sa, B, sb, e):
    sums = (B[e].double() * A.double().unsqueeze(1)).sum(2).float()
    return ((sa.unsqueeze(1) * sb[e]) * sums).to(torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 128), (5, 384), (6, 512), (7, 640), (130, 2048), (9, 2176), (3, 7168), (5, 8192), (7, 16512)])
def test_quantizer_matches_recipe(M, K, dtype):
    rng = np.random.default_rng(M + K)
    x = torch.from_numpy((rng.standard_normal((M, K)) * np.exp(5 * rng.standard_normal((M, 1)))).astype(np.float32))
    x = x.to(dtype)
    x[M - 1] = 0
    x[0, 0] = 3e38 if dtype == torch.float32 else 1.0
    if M > 2:
        x[1] = 1e-39 if dtype == torch.float32 else 0.5
        x[1, ::3] = 7e-41
    q, s = dg.dg_quantize_int8_per_row(x.cuda())
    wq, ws = ref.quantize_int8(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)
    gq, gs = torch.empty_like(q), torch.empty_like(s)
    assert dg.dg_quantize_int8_per_row(x.cuda(), gq, gs)[0] is gq and torch.equal(gq, q) and torch.equal(gs, s)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantizer_marks_rows_that_are_not_finite(bad):
    x = torch.randn(3, 256, device="cuda")
    x[1, 77] = bad
    q, s = dg.dg_quantize_int8_per_row(x)
    assert torch.isnan(s).tolist() == [False, True, False] and int(q[1].abs().max()) == 0


def test_no_rows():
    e = lambda *n: torch.empty(n, dtype=torch.int8, device="cuda")  # noqa: E731
    f = lambda *n: torch.empty(n, device="cuda")  # noqa: E731
    D = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert dg.dg_int8_gemm_nt(e(0, 128), f(0), e(64, 128), f(64), D) is D
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert dg.dg_int8_gemm_grouped_contiguous(e(0, 128), f(0), e(2, 64, 128), f(2, 64), D, none) is D
    assert dg.dg_quantize_int8_per_row(f(0, 128))[0].shape == (0, 128)
