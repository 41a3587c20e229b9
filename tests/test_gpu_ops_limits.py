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
