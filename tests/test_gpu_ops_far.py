"""Adapters that lie beyond 4 GiB of their matrices, where the dense tiles and
the first product of many rows read them (tests/test_ops_forms.py holds the
sizes to these forms)."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import ops_ref as ref
from tests.gpu_util import to_dev
from tests.test_gpu_ops import host, lora_case, lora_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,R,L", [
    (2048, 2048, 128, 10000),   # 5 GiB each; rows as they come
    (8, 32768, 72, 1024)])      # 4.5 GiB of the first matrix; rows grouped by adapter
def test_lora_adapters_past_four_gib_in_dense_tiles(N, K, R, L):
    M = 1540
    c = lora_case(6, M, N, K, R, 1, "fp32")
    c["ids"] = np.where(np.arange(M) % 13 == 5, 0, -1).astype(np.int32)
    c["ids"][700:710] = 0
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else to_dev(v) for n, v in c.items()}
    for n in ("la", "lb", "scaling"):
        whole = torch.zeros((L,) + tuple(d[n].shape[1:]), dtype=d[n].dtype, device="cuda")
        whole[L - 1] = d[n][0]
        d[n] = whole
    assert d["la"].numel() * 2 > 1 << 32
    ids = torch.where(d["ids"] == 0, torch.full_like(d["ids"], L - 1), d["ids"])
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    dg.dg_fp8_gemm_nt_lora(d["A"], d["sa"], d["B"], d["sb"], D, d["x"], d["la"], d["lb"], ids, d["scaling"])
    want, tol = lora_ref(c, "fp32")
    assert (np.abs(host(D) - want) <= tol + ref.BF16 * (np.abs(want) + tol)).all()
