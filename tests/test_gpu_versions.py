"""Buffers that a call writes: a graph that saved one before refuses to go back
with other values in it, as torch's own in-place operations make it."""
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg

pytestmark = pytest.mark.gpu


def half(*n):
    return torch.randn(*n, device="cuda").to(torch.bfloat16)


def ints(*n):
    return torch.zeros(*n, dtype=torch.int32, device="cuda")


def saved_plan():
    """(out, rows, layout, y): a weighted sum whose graph saved the last three."""
    x, ids = half(4, 128), ints(4, 1)
    _, rows, layout, _ = dg.dg_moe_dispatch(x, ids, 1)
    y, w = half(layout.numel(), 128), torch.rand(4, 1, device="cuda", requires_grad=True)
    return dg.dg_moe_unpermute(y, rows, w, layout=layout), rows, layout, y


def codes(M, K):
    return torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.zeros(M, K // 128, device="cuda")


OVERWRITES = {
    "sort into rows": lambda rows, layout, y: dg.dg_moe_sort(ints(4, 1), 1, rows),
    "sort into layout": lambda rows, layout, y: dg.dg_moe_sort(ints(4, 1), 1, None, layout),
    "dispatch into rows": lambda rows, layout, y: dg.dg_moe_dispatch_fp8(half(4, 128), ints(4, 1), 1, rows=rows),
    "dispatch into layout": lambda rows, layout, y: dg.dg_moe_dispatch_int8(half(4, 128), ints(4, 1), 1, layout=layout),
    "dispatch into y": lambda rows, layout, y: dg.dg_moe_dispatch(half(4, 128), ints(4, 1), 1, y),
    "gate into y": lambda rows, layout, y: dg.dg_swiglu(half(128, 256), None, y),
    "gate's gradient into y": lambda rows, layout, y: dg.dg_swiglu_backward(half(128, 128), half(128, 64), None, y),
    "sum into y": lambda rows, layout, y: dg.dg_moe_unpermute(half(4, 128), ints(128, 1), None, y),
    "sum's gradient into y": lambda rows, layout, y: dg.dg_moe_unpermute_backward(half(4, 128), half(128, 128),
                                                                                 torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1), None, None, y),
    "int8 product into y": lambda rows, layout, y: dg.dg_int8_gemm_nt(*dg.dg_quantize_int8_per_row(half(128, 128)),
                                                                      *dg.dg_quantize_int8_per_row(half(128, 128)), y),
    "FP8 product into y": lambda rows, layout, y: dg.dg_fp8_gemm_nt(*codes(128, 128), codes(128, 128)[0], torch.zeros(1, 1, device="cuda"), y),
    "grouped FP8 product into y": lambda rows, layout, y: dg.dg_fp8_gemm_grouped_contiguous(
        *codes(128, 128), codes(128, 128)[0].view(1, 128, 128), torch.zeros(1, 1, 1, device="cuda"), y, ints(128)),
    "router into rows": lambda rows, layout, y: dg.dg_moe_topk(torch.randn(4, 8, device="cuda"), 1, rows),
}


@pytest.mark.parametrize("name", OVERWRITES)
def test_going_back_with_overwritten_values_is_an_error(name):
    out, *saved = saved_plan()
    OVERWRITES[name](*saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_going_back_past_other_writes():
    out, rows, layout, y = saved_plan()
    with torch.inference_mode():
        h = torch.empty(128, 64, dtype=torch.bfloat16, device="cuda")
        dg.dg_swiglu(y, layout, h)
    dg.dg_swiglu(y, layout, h)  # an inference tensor has no version
    dg.dg_moe_sort(ints(4, 1), 1)
    out.sum().backward()
