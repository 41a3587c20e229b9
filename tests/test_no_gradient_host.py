"""How calls that have no gradient say so, on host tensors: the functions that
the quantizing calls go through."""
import warnings

import pytest
import torch

import fp8_block_scaled_gemm_amd as dg


def test_outputs_with_a_float_refuse_a_gradient_without_a_warning():
    x = torch.ones(3, requires_grad=True)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        q, s = dg._no_grad_rows("call", lambda: (torch.zeros(3, dtype=torch.int8), torch.ones(1)), x, None, None)
    assert not q.requires_grad and s.requires_grad
    with pytest.raises(NotImplementedError, match="call has no gradient"):
        s.sum().backward()


def test_outputs_that_are_all_whole_numbers_warn():
    x = torch.ones(3, requires_grad=True)
    whole = lambda: (torch.zeros(3, dtype=torch.uint8), torch.ones(1, dtype=torch.uint8))  # noqa: E731
    with pytest.warns(UserWarning, match="call records no gradient in whole numbers"):
        q, s = dg._no_grad_rows("call", whole, x, None, None)
    assert not q.requires_grad and not s.requires_grad
