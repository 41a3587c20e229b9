"""One decoder layer's linear work at decode time, with the operators around
the FP8 products used together:

  x -> per-token FP8 -> shared projection with each request's own low-rank
  adapter -> residual -> router (top-k experts) -> per-token FP8 -> expert
  layer -> residual

and one training step of the same router, whose gradient comes from
``dg_moe_topk_backward``.  Weights and activations are random.

    python examples/decode_layer.py [--tokens 8] [--hidden 2048] [--inner 768]
                                    [--experts 32] [--topk 4] [--adapters 6] [--steps 50]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_gemm_amd as dg  # noqa: E402


class DecodeLayer:
    """Quantized weights of one layer and the buffers of one batch size."""

    def __init__(self, tokens, hidden, inner, experts, topk, adapters, rank=16, device="cuda", seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        randn = lambda *n: torch.randn(*n, generator=gen, device=device)  # noqa: E731
        block = dg.dg_quantize_fp8_per_block
        self.topk = topk
        self.proj, self.proj_s = block(randn(hidden, hidden) * hidden ** -0.5)
        w13 = [block(randn(2 * inner, hidden) * hidden ** -0.5) for _ in range(experts)]
        w2 = [block(randn(hidden, inner) * inner ** -0.5) for _ in range(experts)]
        self.w13, self.s13 = (torch.stack(t) for t in zip(*w13))
        self.w2, self.s2 = (torch.stack(t) for t in zip(*w2))
        self.router = randn(experts, hidden) * hidden ** -0.5
        self.bias = randn(experts) * 0.05
        self.lora_a = (randn(adapters, rank, hidden) * hidden ** -0.5).to(torch.bfloat16)
        self.lora_b = (randn(adapters, hidden, rank) * 0.1).to(torch.bfloat16)
        self.scaling = torch.full((adapters,), 2.0, device=device)
        # the projection's output and the calls' workspaces, kept for every step
        self.mid = torch.empty(tokens, hidden, dtype=torch.bfloat16, device=device)
        scratch = lambda n: torch.empty(n, dtype=torch.uint8, device=device)  # noqa: E731
        self.lora_ws = scratch(dg.dg_fp8_gemm_nt_lora_workspace(tokens, hidden, hidden, adapters, rank))
        self.moe_ws = scratch(dg.dg_moe_mlp_fp8_workspace(tokens, topk, experts, hidden, inner))

    def logits(self, x):
        return torch.mm(x.float(), self.router.t())

    def __call__(self, x, adapter):
        """x [T][H] bf16, adapter [T] int32 (-1: none) -> [T][H] bf16, expert ids."""
        q, s = dg.dg_quantize_fp8_per_token_bf16(x)
        dg.dg_fp8_gemm_nt_lora(q, s, self.proj, self.proj_s, self.mid, x, self.lora_a, self.lora_b, adapter,
                               self.scaling, self.lora_ws)
        h = x + self.mid
        ids, weights = dg.dg_moe_topk(self.logits(h), self.topk, bias=self.bias, scoring="sigmoid")
        q, s = dg.dg_quantize_fp8_per_token_bf16(h)
        return h + dg.dg_moe_mlp_fp8(q, s, ids, weights, self.w13, self.s13, self.w2, self.s2,
                                     workspace=self.moe_ws), ids


def train_router(layer, x, steps=20, rate=1.0):
    """Pulls the router's weights on these tokens towards a target, by plain
    gradient descent on the router; returns the losses."""
    ids, _ = dg.dg_moe_topk(layer.logits(x), layer.topk)
    target = torch.softmax(torch.arange(layer.topk, device=x.device, dtype=torch.float32), 0).expand(len(x), -1)
    router, losses = layer.router.clone(), []
    for _ in range(steps):
        logits = torch.mm(x.float(), router.t())
        picked = torch.softmax(logits.gather(1, ids.long()), 1)  # renormalized scores of the kept experts
        losses.append(float(((picked - target) ** 2).sum(1).mean()))
        grad = dg.dg_moe_topk_backward(logits, ids, 2.0 * (picked - target))
        router -= (rate / x.shape[1]) * torch.mm(grad.t(), x.float())  # |x|^2 is about H
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 8), ("hidden", 2048), ("inner", 768), ("experts", 32), ("topk", 4),
                        ("adapters", 6), ("steps", 50)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    layer = DecodeLayer(a.tokens, a.hidden, a.inner, a.experts, a.topk, a.adapters)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    adapter = (torch.arange(a.tokens, device="cuda") % (a.adapters + 1) - 1).to(torch.int32)
    eager, ids = layer(x, adapter)
    eager = eager.clone()

    # a decode loop replays one captured graph per step
    static_x, graph = x.clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, _ = layer(static_x, adapter)
    graph.replay()
    torch.cuda.synchronize()
    same = bool(torch.equal(out, eager))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) / a.steps * 1e3
    losses = train_router(layer, x)
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}: {us:.1f} us per layer step, "
          f"graph equals eager: {same}; experts in use {int(torch.unique(ids).numel())}; "
          f"router loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    return {"us": us, "same": same, "out": eager, "losses": losses}


if __name__ == "__main__":
    main()
