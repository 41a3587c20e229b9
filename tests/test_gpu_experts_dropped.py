"""Pairs that a caller drops from a plan after the sort: the sum leaves them
out, and the gradient of their rows is zero, without a layout or with one whose
entries say so."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import experts_ref as ref
from tests.gpu_util import to_dev
from tests.test_gpu_experts import bf16, choices, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_layout", [False, True])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 8), (40, 3, 5, 72), (333, 5, 31, 1416), (1030, 8, 12, 264)])
def test_dropped_pairs_have_no_gradient(T, k, E, H, with_layout):
    rng = np.random.default_rng(T + H)
    rows, layout, _ = ref.sort(choices(rng, T, k, E, "own"), E, dg.dg_moe_sort_rows(T, k, E))
    drop = rng.random(rows.shape) < 0.3
    drop[0, 0] = True
    layout[rows[drop & (rows >= 0)]] = -1
    rows[drop] = -1
    y, g = bf16(rng.standard_normal((layout.size, H))), bf16(rng.standard_normal((T, H)))
    w = to_dev(rng.random(rows.shape).astype(np.float32))
    given = to_dev(layout) if with_layout else None
    out, bound = ref.unpermute(host(y), rows, w.cpu().numpy())
    want, y_bound, want_w, w_bound = ref.unpermute_backward(host(g), host(y), rows, w.cpu().numpy())
    # memory that held NaN before: nothing of it comes back
    torch.full_like(y, float("nan"))
    leaf, leaf_w = y.clone().requires_grad_(), w.clone().requires_grad_()
    got = dg.dg_moe_unpermute(leaf, to_dev(rows), leaf_w, layout=given)
    got.backward(g)
    assert (np.abs(host(got.detach()) - out) <= bound).all()
    assert (np.abs(host(leaf.grad) - want) <= y_bound).all()
    assert (np.abs(leaf_w.grad.cpu().numpy() - want_w) <= w_bound).all()
    named = np.zeros(layout.size, bool)
    named[rows[rows >= 0]] = True
    assert not bool(leaf.grad[to_dev(~named)].any())
