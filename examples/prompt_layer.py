"""One expert layer of a prompt, with the operators around the grouped products
used together:

  x -> router (top-k experts) -> sorted by expert and quantized once per token
  -> grouped product -> gate, quantized -> grouped product -> weighted sum

with FP8 weights (fp32 or power-of-two scales) and with int8 weights, and one
training step of the same layer in bf16, whose gradients come from the same
operators' backward calls through torch's autograd.  Weights and activations
are random.

    python examples/prompt_layer.py [--tokens 2048] [--hidden 2048] [--inner 768]
                                    [--experts 32] [--topk 4] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_gemm_amd as dg  # noqa: E402

FORMS = {  # quantizer of a weight, dispatch, product, gate
    "fp8": (dg.dg_quantize_fp8_per_block, dg.dg_moe_dispatch_fp8, dg.dg_fp8_gemm_grouped_contiguous,
            dg.dg_swiglu_quantize_fp8),
    "e8m0": (dg.dg_quantize_fp8_per_block_e8m0, dg.dg_moe_dispatch_fp8_e8m0, dg.dg_fp8_gemm_grouped_contiguous_e8m0,
             dg.dg_swiglu_quantize_fp8_e8m0),
    "int8": (dg.dg_quantize_int8_per_row, dg.dg_moe_dispatch_int8, dg.dg_int8_gemm_grouped_contiguous,
             dg.dg_swiglu_quantize_int8),
}


def weights_of(experts, hidden, inner, device="cuda", seed=0):
    """Random fp32 weights: router [E][H], gate and up [E][2I][H], down [E][H][I]."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    randn = lambda *n: torch.randn(*n, generator=gen, device=device)  # noqa: E731
    return (randn(experts, hidden) * hidden ** -0.5, randn(experts, 2 * inner, hidden) * hidden ** -0.5,
            randn(experts, hidden, inner) * inner ** -0.5)


class PromptLayer:
    """Quantized weights of one layer and the buffers of one number of tokens."""

    def __init__(self, form, tokens, topk, router, w13, w2):
        quantize, self.dispatch, self.product, self.gate = FORMS[form]
        self.topk, self.router, self.experts = topk, router, w13.shape[0]
        self.w13, self.s13 = (torch.stack(t) for t in zip(*[quantize(w) for w in w13]))
        self.w2, self.s2 = (torch.stack(t) for t in zip(*[quantize(w) for w in w2]))
        rows = dg.dg_moe_sort_rows(tokens, topk, self.experts)
        self.z = torch.empty(rows, w13.shape[1], dtype=torch.bfloat16, device=w13.device)
        self.y = torch.empty(rows, w2.shape[1], dtype=torch.bfloat16, device=w13.device)
        self.ws = torch.empty(max(16, dg.dg_moe_sort_workspace(tokens, topk, self.experts)), dtype=torch.uint8,
                              device=w13.device)

    def __call__(self, x):
        """x [T][H] bf16 -> [T][H] bf16."""
        ids, weights = dg.dg_moe_topk(torch.mm(x.float(), self.router.t()), self.topk)
        a, sa, rows, layout, _ = self.dispatch(x, ids, self.experts, workspace=self.ws)
        self.product(a, sa, self.w13, self.s13, self.z, layout)
        h, sh = self.gate(self.z, layout)
        self.product(h, sh, self.w2, self.s2, self.y, layout)
        return dg.dg_moe_unpermute(self.y, rows, weights)


def train_forward(x, router, w13, w2, topk):
    """The same layer in bf16 with plain products per expert, differentiable in
    every argument: router, sort, gate and sum by this library's operators."""
    ids, weights = dg.dg_moe_topk(torch.mm(x.float(), router.t()), topk)
    a, rows, layout, offsets = dg.dg_moe_dispatch(x, ids, w13.shape[0])
    first = offsets.tolist()  # each expert's rows, whole blocks

    def product(t, w):
        parts = [torch.mm(t[first[e]:first[e + 1]].float(), w[e].t()) for e in range(len(first) - 1)]
        rest = torch.zeros(t.shape[0] - first[-1], w.shape[1], device=t.device)
        return torch.cat(parts + [rest]).to(torch.bfloat16)
    y = product(dg.dg_swiglu(product(a, w13), layout), w2)
    return dg.dg_moe_unpermute(y, rows, weights, layout=layout)


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("hidden", 2048), ("inner", 768), ("experts", 32), ("topk", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    router, w13, w2 = weights_of(a.experts, a.hidden, a.inner)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        plain = train_forward(x, router, w13, w2, a.topk).float()
    got = {"plain": plain}
    for form in FORMS:
        layer = PromptLayer(form, a.tokens, a.topk, router, w13, w2)
        eager = layer(x).clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x)
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
        off = float((eager.float() - plain).norm() / plain.norm())
        print(f"{form}: {a.tokens} tokens, {a.topk} of {a.experts} experts of {a.hidden} x {a.inner}: {us:.1f} us, "
              f"graph equals eager: {same}, off the bf16 layer by {off:.4f}", flush=True)
        got[form] = {"out": eager, "same": same, "us": us, "off": off}
    leaves = [t.clone().requires_grad_() for t in (x, router, w13, w2)]
    out = train_forward(*leaves, a.topk)
    target = torch.randn(a.tokens, a.hidden, device="cuda")
    loss = ((out.float() - target) ** 2).mean()
    loss.backward()
    got["grads"] = [t.grad for t in leaves]
    print("gradient norms of x, router, gate and up, down: " + ", ".join(f"{float(t.grad.float().norm()):.3g}" for t in leaves))
    return got


if __name__ == "__main__":
    main()
