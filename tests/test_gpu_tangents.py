"""A dual tensor's tangent is never dropped: the operators have no forward-mode
derivative, so new outputs refuse it and given ones warn."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import fp8_block_scaled_gemm_amd as dg

pytestmark = pytest.mark.gpu


def half(*n):
    return torch.randn(*n, device="cuda").to(torch.bfloat16)


IDS = lambda: torch.zeros(4, 1, dtype=torch.int32, device="cuda")  # noqa: E731
ROWS = lambda: torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1)  # noqa: E731
CALLS = {  # call of a dual tensor, and that tensor's primal
    "dispatch": (lambda x: dg.dg_moe_dispatch(x, IDS(), 2), lambda: half(4, 256)),
    "dispatch_fp8": (lambda x: dg.dg_moe_dispatch_fp8(x, IDS(), 2), lambda: half(4, 256)),
    "dispatch_e8m0": (lambda x: dg.dg_moe_dispatch_fp8_e8m0(x, IDS(), 2), lambda: half(4, 256)),
    "dispatch_int8": (lambda x: dg.dg_moe_dispatch_int8(x, IDS(), 2), lambda: half(4, 256)),
    "unpermute": (lambda y: dg.dg_moe_unpermute(y, ROWS()), lambda: half(4, 64)),
    "unpermute_weights": (lambda w: dg.dg_moe_unpermute(half(4, 64), ROWS(), w), lambda: torch.rand(4, 1, device="cuda")),
    "swiglu": (dg.dg_swiglu, lambda: half(4, 256)),
    "swiglu_fp8": (dg.dg_swiglu_quantize_fp8, lambda: half(4, 256)),
    "swiglu_e8m0": (dg.dg_swiglu_quantize_fp8_e8m0, lambda: half(4, 256)),
    "swiglu_int8": (dg.dg_swiglu_quantize_int8, lambda: half(4, 256)),
    "quantize_int8": (dg.dg_quantize_int8_per_row, lambda: half(4, 256)),
    "topk": (lambda x: dg.dg_moe_topk(x, 2), lambda: torch.randn(4, 8, device="cuda")),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tangent_is_refused(name):
    call, primal = CALLS[name]
    x = primal()
    call(x)
    with fw.dual_level():
        dual = fw.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError, match="forward mode"):
            call(dual)
        with torch.no_grad(), pytest.raises(NotImplementedError, match="forward mode"):
            call(dual)


def test_a_given_output_warns():
    z, h = half(4, 256), half(4, 128)
    with fw.dual_level():
        with pytest.warns(UserWarning, match="no gradient"):
            dg.dg_swiglu(fw.make_dual(z, torch.ones_like(z)), None, h)
    assert torch.equal(h, dg.dg_swiglu(z))
