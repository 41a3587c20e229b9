"""Forward-mode tangents: the binding sees them, so that no call drops one."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import fp8_block_scaled_gemm_amd as dg
from tests.test_ops_limits import lib  # noqa: F401  (fixture: builds what is missing)


def test_a_tangent_counts_as_a_gradient_that_is_wanted(lib):  # noqa: F811
    wants = dg._ops().wants_grad
    x = torch.zeros(3)
    assert not wants(x) and not wants(None, x, 3)
    with fw.dual_level():
        dual = fw.make_dual(x, torch.ones(3))
        assert wants(dual) and wants(None, x, dual)
        with torch.no_grad():  # which keeps tangents
            assert wants(dual) and not wants(x.requires_grad_())
        with fw._set_fwd_grad_enabled(False):
            assert not wants(dual.detach())
        assert not wants(fw.unpack_dual(dual).primal.detach())
    assert not wants(torch.zeros(3))


@pytest.mark.parametrize("requires", [False, True])
def test_gradients_are_wanted_as_before(lib, requires):  # noqa: F811
    x = torch.zeros(2, requires_grad=requires)
    assert dg._ops().wants_grad(x) is requires
    with torch.no_grad():
        assert not dg._ops().wants_grad(x)
    with torch.inference_mode():
        assert not dg._ops().wants_grad(x, torch.zeros(1))
