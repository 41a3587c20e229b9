"""examples/decode_layer.py: the operators used together, eagerly, from a
captured graph and in a training step."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_layer_example():
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(["--tokens", "5", "--hidden", "512", "--inner", "256", "--experts", "8", "--topk", "2",
                        "--adapters", "3", "--steps", "3"])
    assert got["same"]
    assert got["out"].shape == (5, 512) and bool(torch.isfinite(got["out"]).all())
    losses = got["losses"]
    assert all(b <= a for a, b in zip(losses, losses[1:])) and losses[-1] < 0.5 * losses[0]
