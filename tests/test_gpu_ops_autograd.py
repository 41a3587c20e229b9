"""Gradients through the operators of include/dg_ops.h as torch records them:
the router's weights have one, the others say that they have none."""
import warnings

import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import ops_ref as ref
from tests.gpu_util import to_dev
from tests.test_gpu_ops import MOE_ORDER, host, lora_case, moe_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring,renorm,G", [("softmax", True, 1), ("softmax", False, 4), ("sigmoid", True, 4)])
def test_topk_weights_carry_the_gradient_of_the_logits(scoring, renorm, G, dtype):
    x = torch.randn(37, 64, device="cuda").to(dtype)
    bias = torch.randn(64, device="cuda") * 0.1
    how = dict(scoring=scoring, renormalize=renorm, scale=1.5)
    ids, w = dg.dg_moe_topk(x, 5, bias=bias, n_group=G, topk_group=(G + 1) // 2, **how)
    g = torch.randn(37, 5, device="cuda")
    want = dg.dg_moe_topk_backward(x, ids, g, **how)
    leaf = x.clone().requires_grad_()
    got_ids, got_w = dg.dg_moe_topk(leaf, 5, bias=bias, n_group=G, topk_group=(G + 1) // 2, **how)
    assert torch.equal(got_ids, ids) and torch.equal(got_w, w)
    assert got_w.requires_grad and not got_ids.requires_grad
    (got_w * g).sum().backward()
    assert leaf.grad.dtype == dtype and torch.equal(leaf.grad, want)


def test_topk_gradient_goes_on_to_what_makes_the_logits():
    """Central differences, in 64 bits, of the definition behind a product."""
    rng = np.random.default_rng(6)
    h, r = rng.standard_normal((4, 8)), rng.standard_normal((20, 8))
    gw = rng.standard_normal((4, 3)).astype(np.float32)
    x = to_dev(h.astype(np.float32))
    router = to_dev(r.astype(np.float32)).requires_grad_()
    ids, w = dg.dg_moe_topk(torch.mm(x, router.t()), 3, renormalize=False)
    (w * to_dev(gw)).sum().backward()
    at, step = ids.cpu().numpy(), 1e-5
    h64, r64 = h.astype(np.float32).astype(np.float64), r.astype(np.float32).astype(np.float64)

    def loss(m):
        return (ref.topk_weights(h64 @ m.T, at, "softmax", False, 1.0) * gw).sum()
    want = np.zeros_like(r64)
    for i in np.ndindex(*r64.shape):
        up, down = r64.copy(), r64.copy()
        up[i] += step
        down[i] -= step
        want[i] = (loss(up) - loss(down)) / (2 * step)
    # fp32 logits of |x| up to about 10, their exponentials, and sums over 4 rows
    assert np.abs(host(router.grad) - want).max() <= 1e-8 + 512 * ref.FP32 * np.abs(gw).sum() * np.abs(h).max()


def test_topk_gradient_of_a_constant_and_on_another_stream():
    x = torch.randn(9, 40, device="cuda", requires_grad=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ids, w = dg.dg_moe_topk(x, 4, renormalize=False)
        grad, = torch.autograd.grad(w.sum(), x)  # the gradient arrives expanded, not laid out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(grad, dg.dg_moe_topk_backward(x.detach(), ids, torch.ones_like(w), renormalize=False))


def test_topk_records_nothing_where_nothing_is_asked():
    x = torch.randn(9, 40, device="cuda", requires_grad=True)
    for got in (dg.dg_moe_topk(x.detach(), 4), dg.dg_moe_topk(x.detach(), 4, bias=x[0].detach().requires_grad_())):
        assert not got[1].requires_grad
    with torch.no_grad():
        assert not dg.dg_moe_topk(x, 4)[1].requires_grad
    ids, w = torch.empty(9, 4, dtype=torch.int32, device="cuda"), torch.empty(9, 4, device="cuda")
    with pytest.warns(UserWarning, match="no gradient"):
        assert dg.dg_moe_topk(x, 4, ids, w)[1] is w
    assert not w.requires_grad


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
def test_moe_says_that_it_has_no_gradient(kind):
    d = {n: to_dev(v) for n, v in moe_case(8, 5, 2, 3, 128, 128, kind).items()}
    call = dg.dg_moe_mlp_fp8 if kind == "fp32" else dg.dg_moe_mlp_fp8_e8m0
    plain = call(*[d[n] for n in MOE_ORDER])
    assert not plain.requires_grad
    d["weights"].requires_grad_()
    y = call(*[d[n] for n in MOE_ORDER])
    assert torch.equal(y, plain)
    with pytest.raises(NotImplementedError, match="no gradient"):
        y.sum().backward()
    with torch.no_grad():
        assert not call(*[d[n] for n in MOE_ORDER]).requires_grad
    with pytest.warns(UserWarning, match="no gradient"):
        call(*[d[n] for n in MOE_ORDER], y=torch.empty_like(plain))


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
def test_lora_says_that_it_records_no_gradient(kind):
    c = lora_case(8, 5, 64, 128, 8, 2, kind)
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else to_dev(v) for n, v in c.items()}
    call = dg.dg_fp8_gemm_nt_lora if kind == "fp32" else dg.dg_fp8_gemm_nt_lora_e8m0
    args = ("A", "sa", "B", "sb", "D", "x", "la", "lb", "ids", "scaling")
    d["D"] = torch.empty(5, 64, dtype=torch.bfloat16, device="cuda")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        plain = call(*[d[n] for n in args]).clone()
    for n in ("la", "lb", "scaling", "x"):
        with pytest.warns(UserWarning, match="no gradient"):
            got = call(*[d[m].clone().requires_grad_() if m == n else d[m] for m in args])
        assert torch.equal(got, plain) and not got.requires_grad
