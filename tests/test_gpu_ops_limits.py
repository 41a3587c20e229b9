"""The operators of include/dg_ops.h on the GPU at the ends of their sizes."""
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests.gpu_util import to_dev
from tests.test_gpu_ops import lora_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
def test_lora_no_rows(kind):
    c = lora_case(9, 1, 264, 256, 16, 3, kind)
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else to_dev(v) for n, v in c.items()}
    call = dg.dg_fp8_gemm_nt_lora if kind == "fp32" else dg.dg_fp8_gemm_nt_lora_e8m0
    D = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    got = call(d["A"][:0], d["sa"][:0], d["B"], d["sb"], D, d["x"][:0], d["la"], d["lb"], d["ids"][:0], d["scaling"])
    assert got is D and got.shape == (0, 264)


# A grid holds at most 2^32 - 1 work-items: 2^26 tokens of 64 lanes pass it.
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_topk_and_gradient_of_more_rows_than_one_grid_holds(scoring):
    T = 2 ** 26 + 5
    x = torch.randn(T, 2, device="cuda", dtype=torch.bfloat16)
    ids, w = dg.dg_moe_topk(x, 1, scoring=scoring, renormalize=False)
    g = torch.randn(T, 1, device="cuda")
    dx = dg.dg_moe_topk_backward(x, ids, g, scoring=scoring, renormalize=False)
    step = 2 ** 24
    for r in range(0, T, step):
        a, b = x[r:r + step, 0].float(), x[r:r + step, 1].float()
        second = b > a
        assert torch.equal(ids[r:r + step, 0], second.int())
        p = torch.sigmoid(torch.where(second, b, a) if scoring == "sigmoid" else (a - b).abs())
        # the exponential, a sum and a quotient in 32 bits, on both sides
        assert bool(((w[r:r + step, 0] - p).abs() <= 64 * 2.0 ** -24 * p).all())
        d = g[r:r + step, 0] * p * (1 - p)
        want = torch.stack([torch.where(second, 0 * d if scoring == "sigmoid" else -d, d),
                            torch.where(second, d, 0 * d if scoring == "sigmoid" else -d)], 1)
        err = (dx[r:r + step].float() - want).abs()
        assert bool((err <= 2.0 ** -8 * want.abs() + 256 * 2.0 ** -24 * g[r:r + step].abs()).all())
