"""The operators of include/dg_ops.h where other code paths take over: many
rows beside the dense tiles, experts numbered by pair, weights past 4 GiB."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import ops_ref as ref
from tests.gpu_util import to_dev
from tests.test_gpu_ops import (INF, MOE_ORDER, NAN, check_lora, check_moe, host, lora_case, lora_ref, moe_case,
                                run_lora)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("T,k,E,H,I", [(12, 2, 30, 128, 2048), (20, 2, 64, 128, 128), (66, 1, 90, 128, 256),
                                       (2, 8, 20, 384, 2048), (16, 8, 12, 256, 256), (100, 3, 4, 256, 128)])
def test_moe_other_paths(T, k, E, H, I, kind):
    check_moe(moe_case(T + E, T, k, E, H, I, kind), kind)


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("M,N,K,R,L,rows", [
    (513, 128, 640, 128, 3, "runs"), (600, 520, 384, 24, 4, "runs"), (700, 264, 128, 8, 5, "mixed"),
    (1030, 392, 256, 72, 7, "mixed"), (600, 136, 256, 40, 64, "each"), (530, 8, 128, 64, 600, "each"),
    (520, 256, 1152, 16, 2, "none")])
def test_lora_many_rows(M, N, K, R, L, rows, kind):
    check_lora(lora_case(M + N, M, N, K, R, L, kind, rows), kind)


@pytest.mark.parametrize("shape", ["256x256", "256x224", "256x192", "256x160", "128x256", "128x128",
                                   "128x64", "128x32", "256x256t"])
def test_lora_every_dense_tile_shape(shape, monkeypatch):
    monkeypatch.setenv("DG_FP8_DENSE_TILE", shape)
    kind = "e8m0" if shape.endswith("t") else "fp32"
    check_lora(lora_case(3, 600, 328, 256, 72, 5, kind, "mixed"), kind)


def test_lora_infinities_stay_in_their_rows_of_a_dense_tile():
    c = lora_case(11, 600, 136, 256, 16, 4, "fp32", "each")
    c["la"][1, 3, 7] = INF
    c["lb"][2] = NAN
    c["scaling"][3] = INF
    c["x"][5, 9] = NAN
    c["ids"][5] = -1
    clean = np.isin(c["ids"], [-1, 0])
    check_lora(c, "fp32", rows=clean)
    got = host(run_lora(c, "fp32"))
    assert np.isnan(got[c["ids"] == 2]).all()
    assert not np.isfinite(got[c["ids"] == 3]).any()


def test_lora_many_rows_graph_and_stream():
    c = lora_case(23, 600, 264, 256, 24, 3, "fp32", "runs")
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else to_dev(v) for n, v in c.items()}
    D = torch.empty(600, 264, dtype=torch.bfloat16, device="cuda")
    call = lambda out: dg.dg_fp8_gemm_nt_lora(  # noqa: E731
        d["A"], d["sa"], d["B"], d["sb"], out, d["x"], d["la"], d["lb"], d["ids"], d["scaling"])
    eager = call(torch.empty_like(D))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(D)
    for _ in range(3):
        D.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D, eager)
        call(torch.empty_like(D))
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(torch.empty_like(D))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, eager)


def test_moe_weights_past_four_gib():
    """The experts in use lie beyond 4 GiB of both weights."""
    E, H, I = 600, 2048, 4096           # 10 GiB and 5 GiB; only the experts in use are set
    small = moe_case(5, 3, 2, 2, H, I, "fp32")
    at = [E - 1, E - 3]
    d = {n: to_dev(small[n]) for n in ("x", "sx", "weights")}
    for n in ("w13", "s13", "w2", "s2"):
        t = to_dev(small[n])
        whole = torch.zeros((E,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
        for i, e in enumerate(at):
            whole[e] = t[i]
        d[n] = whole
    d["ids"] = to_dev(np.array(at, np.int32)[small["ids"]])
    got = host(dg.dg_moe_mlp_fp8(*[d[n] for n in MOE_ORDER]))
    want, tol = ref.moe(*[small[n] for n in MOE_ORDER], "fp32")
    assert (np.abs(got - want) <= tol + ref.BF16 * (np.abs(want) + tol)).all()


@pytest.mark.parametrize("M", [3, 520])
def test_lora_adapters_past_four_gib(M):
    """The adapter in use lies beyond 4 GiB of both matrices."""
    L, N, K, R = 10000, 2048, 2048, 128     # 5 GiB each
    c = lora_case(6, M, N, K, R, 1, "fp32")
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else to_dev(v) for n, v in c.items()}
    for n in ("la", "lb", "scaling"):
        whole = torch.zeros((L,) + tuple(d[n].shape[1:]), dtype=d[n].dtype, device="cuda")
        whole[L - 1] = d[n][0]
        d[n] = whole
    ids = torch.where(d["ids"] == 0, torch.full_like(d["ids"], L - 1), d["ids"])
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    dg.dg_fp8_gemm_nt_lora(d["A"], d["sa"], d["B"], d["sb"], D, d["x"], d["la"], d["lb"], ids, d["scaling"])
    want, tol = lora_ref(c, "fp32")
    assert (np.abs(host(D) - want) <= tol + ref.BF16 * (np.abs(want) + tol)).all()


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("M,N,K,R,L,rows", [
    (65, 136, 256, 128, 2, "mixed"), (70, 40, 128, 8, 1024, "each"), (70, 40, 128, 8, 1025, "each"),
    (515, 72, 384, 24, 16, "mixed"), (1535, 136, 640, 72, 36, "each"), (1537, 136, 256, 40, 64, "each"),
    (1601, 264, 128, 16, 900, "mixed"), (2050, 48, 256, 104, 16, "runs"), (1000, 64, 128, 16, 40, "none")])
def test_lora_rows_grouped_by_adapter(M, N, K, R, L, rows, kind):
    check_lora(lora_case(2 * M + N, M, N, K, R, L, kind, rows), kind)


@pytest.mark.parametrize("M,L", [(8189, 1024), (8192, 5), (8193, 5)])
def test_lora_the_most_rows_that_are_grouped(M, L):
    check_lora(lora_case(M, M, 40, 128, 8, L, "fp32", "mixed"), "fp32")


def test_lora_grouping_passes_over_rows_of_no_adapter():
    c = lora_case(31, 700, 72, 256, 32, 6, "fp32", "each")
    c["ids"][::2] = -1
    c["ids"][1::10] = 6         # past the last adapter: none either
    c["ids"][3::10] = 2 ** 31 - 1
    c["ids"][5:40] = 5
    check_lora(c, "fp32")


@pytest.mark.parametrize("shape", ["256x256", "256x224", "256x192", "256x160", "128x256", "128x128",
                                   "128x64", "128x32", "256x256t"])
def test_lora_every_dense_tile_shape_past_the_few_row_form(shape, monkeypatch):
    monkeypatch.setenv("DG_FP8_DENSE_TILE", shape)
    kind = "e8m0" if shape.endswith("t") else "fp32"
    check_lora(lora_case(3, 1540, 328, 256, 72, 5, kind, "mixed"), kind)


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("M,N,K,R,L,rows", [
    (33, 4096, 128, 128, 1, "mixed"), (50, 3000, 128, 128, 4, "each"), (160, 1032, 256, 128, 3, "runs"),
    (257, 1032, 384, 72, 2, "mixed"), (1540, 136, 256, 40, 64, "each"), (1552, 264, 640, 24, 6, "runs"),
    (1537, 8, 128, 64, 600, "each"), (1600, 256, 1152, 16, 2, "none")])
def test_lora_dense_tiles(M, N, K, R, L, rows, kind):
    check_lora(lora_case(M + 3 * N, M, N, K, R, L, kind, rows), kind)


def test_lora_infinities_stay_in_their_rows_past_the_few_row_form():
    c = lora_case(11, 1540, 136, 256, 16, 4, "fp32", "each")
    c["la"][1, 3, 7] = INF
    c["lb"][2] = NAN
    c["scaling"][3] = INF
    c["x"][5, 9] = NAN
    c["ids"][5] = -1
    clean = np.isin(c["ids"], [-1, 0])
    check_lora(c, "fp32", rows=clean)
    got = host(run_lora(c, "fp32"))
    assert np.isnan(got[c["ids"] == 2]).all()
    assert not np.isfinite(got[c["ids"] == 3]).any()


def test_lora_dense_tiles_graph_and_stream():
    c = lora_case(23, 1540, 264, 256, 24, 3, "fp32", "runs")
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else to_dev(v) for n, v in c.items()}
    D = torch.empty(1540, 264, dtype=torch.bfloat16, device="cuda")
    call = lambda out: dg.dg_fp8_gemm_nt_lora(  # noqa: E731
        d["A"], d["sa"], d["B"], d["sb"], out, d["x"], d["la"], d["lb"], d["ids"], d["scaling"])
    eager = call(torch.empty_like(D))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(D)
    for _ in range(3):
        D.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D, eager)
        call(torch.empty_like(D))
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(torch.empty_like(D))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, eager)
