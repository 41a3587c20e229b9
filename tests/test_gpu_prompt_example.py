"""examples/prompt_layer.py: its three forms, eagerly and from captured graphs,
and the gradients of its training step against plain autograd in 64 bits."""
import importlib.util
import os

import pytest
import torch

from tests.experts_ref import BF16

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("prompt_layer", os.path.join(ROOT, "examples", "prompt_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_prompt_layer_example_runs(example):
    got = example.main(["--tokens", "300", "--hidden", "512", "--inner", "256", "--experts", "8", "--topk", "2",
                        "--steps", "2"])
    for form in ("fp8", "e8m0", "int8"):
        assert got[form]["same"] and got[form]["out"].shape == (300, 512)
        # three values are rounded to codes on the way (activations, weights and hidden values, of which each
        # counts once in either product): half a step of e4m3 is at most 2^-4 of a value, of int8 1/254 of a row's
        # largest, which is below 2^-4 of its root mean square (512 normal values: their largest is below 5)
        assert got[form]["off"] <= 4 * 2.0 ** -4
    assert all(bool(torch.isfinite(g.float()).all()) for g in got["grads"])


def test_training_step_gradients(example):
    T, H, I, E, k = 70, 64, 48, 5, 2
    router, w13, w2 = example.weights_of(E, H, I, seed=2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
    g = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
    leaves = [t.clone().requires_grad_() for t in (x, router, w13, w2)]
    example.train_forward(*leaves, k).backward(g)
    x64, r64, a64, b64 = (t.detach().double().requires_grad_() for t in leaves)
    logits = x64 @ r64.t()
    ids = torch.topk(logits, k).indices
    p = torch.softmax(logits, 1).gather(1, ids)
    p = p / p.sum(1, keepdim=True)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        z = x64[t] @ a64[e].t()
        h = z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]
        out = out.index_add(0, t, (h @ b64[e].t()) * p[t, j][:, None])
    out.backward(g.double())
    # the step rounds eight tensors to bf16 on the way (rows, z, h, y, their gradients, the sum of x's two), each by
    # at most 2^-8 of its values; the products' norms are about one
    for leaf, want in zip(leaves, (x64, r64, a64, b64)):
        assert float((leaf.grad.double() - want.grad).norm() / want.grad.norm()) <= 8 * BF16
