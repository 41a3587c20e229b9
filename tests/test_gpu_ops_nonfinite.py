"""Infinities, NaN and the largest numbers in the operators of
include/dg_ops.h: the results are those of the definition, whichever form the
sizes choose."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import ops_ref as ref
from tests.gpu_util import to_dev
from tests.test_gpu_ops import INF, NAN, host, lora_case, lora_ref, run_lora

pytestmark = pytest.mark.gpu


def _nonfinite_case(M, R, kind, N=136, K=256):
    """Adapter 1: one infinite entry of the rank vector; 2: infinities in the
    second matrix; 3: an entry past the largest bf16, which is finite; 4: an
    infinite entry times zeros; 5: NaN scaling; 0 and rows of none: finite."""
    c = lora_case(17, M, N, K, R, 6, kind, "each")
    c["x"][:, 0] = 1.0
    c["la"][1, 3, 7] = INF
    c["lb"][1, :, 3] = torch.where(c["lb"][1, :, 3] == 0, torch.ones(N, dtype=torch.bfloat16), c["lb"][1, :, 3])
    c["lb"][2, 5, R - 4] = INF
    c["lb"][2, 6, 1] = -INF
    c["la"][3] = 0
    c["la"][3, R - 3, 0] = 1.0
    c["scaling"][3] = 3.3999e38           # rounds to infinity in bf16
    c["lb"][3] = c["lb"][3].float().mul(2.0 ** -124).to(torch.bfloat16)
    c["la"][4, 2, 5] = -INF
    c["lb"][4, ::2, 2] = 0
    c["scaling"][5] = NAN
    return c


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("M,R", [(20, 24), (20, 104), (300, 24), (1540, 24), (1540, 104)])
def test_lora_nonfinite_values_follow_the_definition(M, R, kind):
    c = _nonfinite_case(M, R, kind)
    with np.errstate(all="ignore"):
        want, tol = lora_ref(c, kind)
    got = host(run_lora(c, kind))
    for special in (np.isnan, np.isposinf, np.isneginf):
        bad = special(got) != special(want)
        assert not bad.any(), f"{special.__name__}: adapters {np.unique(c['ids'][np.argwhere(bad)[:, 0]])}"
    fin = np.isfinite(want)
    assert np.isposinf(want).any() and np.isneginf(want).any() and fin[c["ids"] == 3].all()
    # an element whose own terms are finite has a finite bound
    row, col = np.argwhere(fin).T
    assert (np.abs(got[row, col] - want[row, col])
            <= tol[row, col] + ref.BF16 * (np.abs(want[row, col]) + tol[row, col]) + 1e-37).all()


@pytest.mark.parametrize("shape", ["256x256", "256x224", "256x192", "256x160", "128x256", "128x128",
                                   "128x64", "128x32", "256x256t"])
def test_lora_nonfinite_values_in_every_dense_tile(shape, monkeypatch):
    monkeypatch.setenv("DG_FP8_DENSE_TILE", shape)
    test_lora_nonfinite_values_follow_the_definition(1540, 72, "e8m0" if shape.endswith("t") else "fp32")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_topk_backward_masked_experts_get_zero_beside_a_nonfinite_gradient(value, scoring, renorm, dtype):
    rng = np.random.default_rng(3)
    T, E, k = 6, 70, 3
    x = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    x[:, 5:40] = -INF
    x[:, 50] = NAN
    x = x.to(dtype).cuda()
    ids, _ = dg.dg_moe_topk(x, k)
    gw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    clean = dg.dg_moe_topk_backward(x, ids, gw, scoring=scoring, renormalize=renorm)
    gw[1, 1] = value
    got = dg.dg_moe_topk_backward(x, ids, gw, scoring=scoring, renormalize=renorm)
    masked = ~(x > -INF)
    assert bool((got[masked] == 0).all())
    assert not bool(torch.isfinite(got[1]).all())
    others = torch.arange(T, device="cuda") != 1
    assert torch.equal(got[others], clean[others])


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_topk_backward_passes_over_a_masked_expert_that_is_listed(scoring, renorm):
    """Its weight is 0 whatever its gradient: as if the entry were -1."""
    x = torch.randn(3, 20, device="cuda")
    x[:, 4] = -INF
    x[:, 9] = NAN
    ids = torch.tensor([[1, 4, 9], [4, 2, 3], [9, 7, 4]], dtype=torch.int32, device="cuda")
    gw = torch.randn(3, 3, device="cuda")
    gw[0, 1], gw[1, 0], gw[2, 0] = INF, NAN, -INF
    got = dg.dg_moe_topk_backward(x, ids, gw, scoring=scoring, renormalize=renorm)
    skipped = torch.where((ids == 4) | (ids == 9), torch.full_like(ids, -1), ids)
    assert torch.equal(got, dg.dg_moe_topk_backward(x, skipped, gw, scoring=scoring, renormalize=renorm))
    assert bool(torch.isfinite(got).all())
