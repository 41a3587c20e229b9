"""Every quantizing call of include/dg_experts.h and include/dg_int8.h whose
input requires a gradient refuses to pass one back, or warns where it cannot."""
import warnings

import pytest
import torch

import fp8_block_scaled_gemm_amd as dg

pytestmark = pytest.mark.gpu


def run(name, x):
    ids = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    call = getattr(dg, name)
    return call(x, ids, 2) if "dispatch" in name else call(x)


@pytest.mark.parametrize("name", ["dg_moe_dispatch_fp8", "dg_moe_dispatch_int8", "dg_swiglu_quantize_fp8",
                                  "dg_swiglu_quantize_int8", "dg_quantize_int8_per_row"])
def test_scales_in_fp32_refuse(name):
    x = torch.randn(4, 256, device="cuda").to(torch.bfloat16).requires_grad_()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        got = run(name, x)
    assert got[1].requires_grad and not got[0].requires_grad
    with pytest.raises(NotImplementedError, match="no gradient"):
        got[1].sum().backward()
    assert x.grad is None


@pytest.mark.parametrize("name", ["dg_moe_dispatch_fp8_e8m0", "dg_swiglu_quantize_fp8_e8m0"])
def test_scales_in_bytes_warn(name):
    x = torch.randn(4, 256, device="cuda").to(torch.bfloat16).requires_grad_()
    with pytest.warns(UserWarning, match=f"{name} records no gradient"):
        got = run(name, x)
    assert not any(t.requires_grad for t in got)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            run(name, x)
        run(name, x.detach())
