"""Measured cases of the expert layer for many tokens around the grouped
products (include/dg_experts.h) and of the 8-bit integer products
(include/dg_int8.h): tokens sorted by expert and copied into their experts'
rows, the weighted rows added up per token with the gradient, the gated
activation between an expert's two products with its gradient, and products of
int8 operands with a scale per row on either side.

Every operator is given here in its plain form too: elementary torch
operations in 32 bits, rounded once at the end.  ``run`` takes the plain form
or, with ``own``, the framework's entry points.  Rows that belong to no expert
keep what the caller's buffers hold (zeros here) where the outputs are codes
or a product's rows, and are zeros in copied bf16 rows and in gradients.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
BLOCK = 128  # rows that an expert's rows are padded to


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token, 256 experts of which 8 are chosen: rows of its own for each, bound by latency
        dict(name="dispatch_token", op="dispatch", T=1, E=256, k=8, H=7168, local=1.0, to="fp8"),
        # a prompt: the activations quantized once and copied to eight experts each
        dict(name="dispatch_prompt", op="dispatch", T=4096, E=256, k=8, H=7168, local=1.0, to="fp8"),
        # a ragged micro-batch in bf16 (training), half of the experts on another GPU
        dict(name="dispatch_odd", op="dispatch", T=333, E=31, k=5, H=1416, local=0.5, to="bf16"),
        # a decode batch's weighted sum, some pairs elsewhere
        dict(name="combine_odd", op="combine", T=61, E=20, k=6, H=1032, local=0.5),
        # a prompt's weighted sum
        dict(name="combine_prompt", op="combine", T=4096, E=256, k=8, H=7168, local=1.0),
        # the gradients of a prompt's weighted sum: rows and weights
        dict(name="combine_grad_prompt", op="combine_grad", T=4096, E=256, k=8, H=7168, local=1.0),
        # the same for a ragged last micro-batch of a small layer
        dict(name="combine_grad_odd", op="combine_grad", T=777, E=12, k=3, H=904, local=1.0),
        # between a prompt's two products: 256 experts' rows, their padding skipped
        dict(name="gate_prompt", op="gate", T=4096, E=256, k=8, I=2048, local=1.0),
        # its gradient, one expert in four on this GPU
        dict(name="gate_grad_spread", op="gate_grad", T=4096, E=16, k=4, I=1408, local=0.25),
        # one decoded token through an int8 projection
        dict(name="int8_token", op="int8", M=1, N=7168, K=2048),
        # a prompt through the same projection
        dict(name="int8_prompt", op="int8", M=4096, N=7168, K=2048),
        # a prompt's rows of eight experts on this GPU, out of 64, int8 weights
        dict(name="int8_experts", op="int8_grouped", T=4096, E=8, k=8, local=0.125, N=4096, K=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(("dispatch", "combine", "combine_grad", "gate", "gate_grad", "int8", "int8", "int8_grouped"))
    if op == "int8":
        N, K = 8 * _log(rng, 16, 896), 128 * _log(rng, 1, 56)
        return dict(op=op, M=min(_log(rng, 1, 4096), 60_000_000_000 // (N * K)), N=N, K=K)
    c = dict(op=op, T=_log(rng, 1, 4096), E=_log(rng, 2, 256), local=rng.choice((1.0, 0.5, 0.125)))
    c["k"] = rng.randint(1, min(8, c["E"]))
    if op == "int8_grouped":
        c.update(E=min(c["E"], 16), N=8 * _log(rng, 16, 512), K=128 * _log(rng, 1, 56))
        c.update(k=min(c["k"], c["E"]), T=min(c["T"], 512))
    elif op == "dispatch":
        c["to"] = rng.choice(("fp8", "fp8", "bf16"))
        c["H"] = 128 * _log(rng, 1, 56) if c["to"] == "fp8" else 8 * _log(rng, 16, 896)
    elif op in ("combine", "combine_grad"):
        c["H"] = 8 * _log(rng, 16, 896)
    else:
        c["I"] = 128 * _log(rng, 1, 16)
    return c


# --------------------------------------------------------- inputs of the cases

def _capacity(c):
    """Rows that hold every expert's rows padded to whole blocks, whatever the choice of experts."""
    P = c["T"] * c["k"]
    return (P + (BLOCK - 1) * min(c["E"], P)) // BLOCK * BLOCK


def _ids(c, gen):
    """k different experts a token out of the whole layer's; -1 for those on other GPUs."""
    spread = max(c["E"], c["k"], int(round(c["E"] / c["local"])))  # the first E of them are here
    ids = torch.rand(c["T"], spread, generator=gen, device=DEV).argsort(1)[:, :c["k"]]
    return torch.where(ids < c["E"], ids, torch.full_like(ids, -1)).to(torch.int32).contiguous()


def _int8_rows(x):
    s = x.abs().amax(-1, keepdim=True) / 127.0
    q = torch.where(s > 0, (x / s).round(), torch.zeros_like(x)).to(torch.int8)
    return q, s.squeeze(-1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    randn = lambda *n: torch.randn(*n, generator=gen, device=DEV)  # noqa: E731
    c, s = dict(case), {"case": dict(case)}
    if c["op"] == "int8":
        s["A"], s["sa"] = _int8_rows(randn(c["M"], c["K"]))
        s["B"], s["sb"] = _int8_rows(randn(c["N"], c["K"]) * c["K"] ** -0.5)
        s["D"] = torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device=DEV)
        return s
    R = _capacity(c)
    ids = _ids(c, gen)
    if c["op"] == "dispatch":
        s["ids"], s["x"] = ids, randn(c["T"], c["H"]).to(torch.bfloat16)
        if c["to"] == "fp8":
            s["q"] = torch.zeros(R, c["H"], dtype=torch.uint8, device=DEV)
            s["s"] = torch.zeros(R, c["H"] // 128, device=DEV)
        return s
    s["rows"], s["layout"], _ = _sort_plain(ids, c)
    if c["op"] in ("combine", "combine_grad"):
        s["y"] = randn(R, c["H"]).to(torch.bfloat16)
        w = torch.exp(randn(c["T"], c["k"]))
        s["weights"] = (w / w.sum(1, keepdim=True)).contiguous()
        if c["op"] == "combine_grad":
            s["grad"] = randn(c["T"], c["H"]).to(torch.bfloat16)
    elif c["op"] in ("gate", "gate_grad"):
        s["z"] = (randn(R, 2 * c["I"]) * 1.5).to(torch.bfloat16)
        if c["op"] == "gate":
            s["q"] = torch.zeros(R, c["I"], dtype=torch.uint8, device=DEV)
            s["s"] = torch.zeros(R, c["I"] // 128, device=DEV)
        else:
            s["grad"] = randn(R, c["I"]).to(torch.bfloat16)
    else:
        s["A"], s["sa"] = _int8_rows(randn(R, c["K"]))
        s["B"], s["sb"] = _int8_rows(randn(c["E"], c["N"], c["K"]) * c["K"] ** -0.5)
        s["D"] = torch.zeros(R, c["N"], dtype=torch.bfloat16, device=DEV)
    return s


def work(case):
    c = case
    if c["op"] == "int8":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + M * N * 2 + 4 * (M + N), "flops": 2 * M * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    spread = max(E, k, int(round(E / c["local"])))
    pairs = T * k * E // spread  # rows that this GPU's experts get, on average
    R = _capacity(c)
    if c["op"] == "dispatch":
        H = c["H"]
        row = H * (1 + 4 / 128) if c["to"] == "fp8" else 2 * H
        return {"bytes": int(T * H * 2 + pairs * row + T * k * 8 + R * 4), "flops": 2 * T * H}
    if c["op"] == "combine":
        return {"bytes": pairs * c["H"] * 2 + T * c["H"] * 2 + T * k * 8, "flops": 2 * pairs * c["H"]}
    if c["op"] == "combine_grad":
        return {"bytes": 2 * pairs * c["H"] * 2 + T * c["H"] * 2 + T * k * 12, "flops": 3 * pairs * c["H"]}
    if c["op"] == "gate":
        return {"bytes": int(pairs * c["I"] * (4 + 1 + 4 / 128) + R * 4), "flops": 8 * pairs * c["I"]}
    if c["op"] == "gate_grad":
        return {"bytes": pairs * c["I"] * (4 + 2 + 4) + R * 4, "flops": 12 * pairs * c["I"]}
    active = E * (1.0 - (1.0 - k / spread) ** T)
    return {"bytes": int(pairs * (c["K"] + 2 * c["N"] + 4) + active * c["N"] * (c["K"] + 4) + R * 4),
            "flops": 2 * pairs * c["N"] * c["K"]}


# ------------------------------------------------------------- the plain forms

def _sort_plain(ids, c):
    """Row of each pair (-1: no expert here), expert of each row (-1: padding), first row of each expert."""
    E, R = c["E"], _capacity(c)
    key = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E)).flatten().long()
    order = torch.sort(key, stable=True)
    count = (order.values.view(1, -1) == torch.arange(E + 1, device=ids.device).view(-1, 1)).sum(1)
    first = torch.cumsum(count, 0) - count  # of each expert, in the order
    padded = (count[:E] + BLOCK - 1) // BLOCK * BLOCK
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(padded, 0)
    within = torch.arange(key.numel(), device=ids.device) - first[order.values]
    start = torch.where(order.values < E, offsets[order.values] + within, torch.full_like(within, -1))
    rows = torch.empty_like(start)
    rows[order.indices] = start
    layout = torch.full((R + 1,), -1, dtype=torch.int32, device=ids.device)
    at = torch.where(rows >= 0, rows, torch.full_like(rows, R))
    layout[at] = torch.where(rows >= 0, key, torch.full_like(key, -1)).to(torch.int32)
    return rows.view(ids.shape).to(torch.int32), layout[:R].contiguous(), offsets.to(torch.int32)


def _codes_plain(x):
    """e4m3 values of x [..., K] over one scale per 128 columns, and the scales."""
    b = x.unflatten(-1, (-1, 128))
    s = b.abs().amax(-1) / 448.0
    d = s.unsqueeze(-1)
    q = torch.where(d > 0, b / d, torch.zeros_like(b)).to(torch.float8_e4m3fn)
    return q.flatten(-2), s


def _dispatch_plain(s, c):
    rows, layout, offsets = _sort_plain(s["ids"], c)
    R, at = layout.numel(), rows.flatten().long()
    at = torch.where(at >= 0, at, torch.full_like(at, R))
    token = torch.arange(c["T"], device=at.device).repeat_interleave(c["k"])
    if c["to"] == "bf16":
        out = torch.zeros(R + 1, c["H"], dtype=torch.bfloat16, device=at.device)
        out[at] = s["x"][token]
        out[R] = 0
        return out[:R], rows, layout, offsets
    q, scale = _codes_plain(s["x"].float())
    oq = torch.zeros(R + 1, c["H"], dtype=torch.uint8, device=at.device)
    os_ = torch.zeros(R + 1, c["H"] // 128, device=at.device)
    oq[at] = q.view(torch.uint8)[token]
    os_[at] = scale[token]
    return oq[:R].view(torch.float8_e4m3fn), os_[:R], rows, layout, offsets


def _combine_plain(s, c):
    rows = s["rows"].long()
    y = s["y"][rows.clamp(min=0)].float()
    w = torch.where(rows >= 0, s["weights"], torch.zeros_like(s["weights"]))
    return (y * w.unsqueeze(2)).sum(1).to(torch.bfloat16)


def _combine_grad_plain(s, c):
    rows, R = s["rows"].long(), s["y"].shape[0]
    here = rows >= 0
    g = s["grad"].float().unsqueeze(1)
    grad_weights = torch.where(here, (s["y"][rows.clamp(min=0)].float() * g).sum(2), torch.zeros_like(s["weights"]))
    grad_y = torch.zeros(R + 1, c["H"], dtype=torch.bfloat16, device=g.device)
    grad_y[torch.where(here, rows, torch.full_like(rows, R)).flatten()] = \
        (g * s["weights"].unsqueeze(2)).to(torch.bfloat16).flatten(0, 1)
    return grad_y[:R], grad_weights


def _gate_plain(s, c):
    z, I = s["z"].float(), c["I"]
    h = z[:, :I] / (1.0 + torch.exp(-z[:, :I])) * z[:, I:]
    h = torch.where((s["layout"] >= 0).unsqueeze(1), h, torch.zeros_like(h))
    return _codes_plain(h)


def _gate_grad_plain(s, c):
    z, I, d = s["z"].float(), c["I"], s["grad"].float()
    g, u = z[:, :I], z[:, I:]
    p = 1.0 / (1.0 + torch.exp(-g))
    out = torch.cat((d * u * p * (1.0 + g * (1.0 - p)), d * g * p), 1)
    return torch.where((s["layout"] >= 0).unsqueeze(1), out, torch.zeros_like(out)).to(torch.bfloat16)


def _int8_plain(s, c):
    sums = torch.matmul(s["A"].float(), s["B"].float().T)
    return (sums * (s["sa"].unsqueeze(1) * s["sb"])).to(torch.bfloat16)


def _int8_grouped_plain(s, c):
    out, first = torch.zeros_like(s["D"]), 0
    experts = torch.arange(c["E"], dtype=torch.int32, device=out.device).view(-1, 1)
    for e, n in enumerate((s["layout"] == experts).sum(1).tolist()):  # the host needs each expert's rows
        r = slice(first, first + n)
        sums = torch.matmul(s["A"][r].float(), s["B"][e].float().T)
        out[r] = (sums * (s["sa"][r].unsqueeze(1) * s["sb"][e])).to(torch.bfloat16)
        first += (n + BLOCK - 1) // BLOCK * BLOCK
    return out


PLAIN = {"dispatch": _dispatch_plain, "combine": _combine_plain, "combine_grad": _combine_grad_plain,
         "gate": _gate_plain, "gate_grad": _gate_grad_plain, "int8": _int8_plain, "int8_grouped": _int8_grouped_plain}


def run(state):
    c, s = state["case"], state
    if not own:
        return PLAIN[c["op"]](s, c)
    import fp8_block_scaled_gemm_amd as dg
    if c["op"] == "dispatch":
        if c["to"] == "bf16":
            return dg.dg_moe_dispatch(s["x"], s["ids"], c["E"])
        q, scale, rows, layout, offsets = dg.dg_moe_dispatch_fp8(s["x"], s["ids"], c["E"], s["q"], s["s"])
        return q.view(torch.float8_e4m3fn), scale, rows, layout, offsets
    if c["op"] == "combine":
        return dg.dg_moe_unpermute(s["y"], s["rows"], s["weights"])
    if c["op"] == "combine_grad":
        return dg.dg_moe_unpermute_backward(s["grad"], s["y"], s["rows"], s["weights"], s["layout"])
    if c["op"] == "gate":
        q, scale = dg.dg_swiglu_quantize_fp8(s["z"], s["layout"], s["q"], s["s"])
        return q.view(torch.float8_e4m3fn), scale
    if c["op"] == "gate_grad":
        return dg.dg_swiglu_backward(s["z"], s["grad"], s["layout"])
    if c["op"] == "int8":
        return dg.dg_int8_gemm_nt(s["A"], s["sa"], s["B"], s["sb"], s["D"])
    return dg.dg_int8_gemm_grouped_contiguous(s["A"], s["sa"], s["B"], s["sb"], s["D"], s["layout"])


# ------------------------------------------------------ the definition, 64 bits

def _sort64(ids, c):
    """By an ordinary loop over the pairs, on the host."""
    ids = ids.cpu().numpy()
    mine = [[] for _ in range(c["E"])]
    for p, e in enumerate(ids.ravel().tolist()):
        if 0 <= e < c["E"]:
            mine[e].append(p)
    rows, layout = np.full(ids.size, -1, np.int32), np.full(_capacity(c), -1, np.int32)
    offsets = [0]
    for e, pairs in enumerate(mine):
        for i, p in enumerate(pairs):
            rows[p], layout[offsets[e] + i] = offsets[e] + i, e
        offsets.append(offsets[e] + -(-len(pairs) // BLOCK) * BLOCK)
    put = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
    return put(rows).view(ids.shape), put(layout), put(offsets)


def _ratio64(v):
    """v [rows, K] over each 128 columns' largest magnitude / 448, and that scale."""
    top = torch.stack([b.abs().max(1).values for b in v.split(128, 1)], 1) / 448
    wide = top.repeat_interleave(128, 1)
    return torch.where(wide > 0, v / wide.clamp(min=1e-300), torch.zeros_like(v)), top


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "dispatch":
        rows, layout, offsets = _sort64(s["ids"], c)
        t, j = torch.nonzero(rows >= 0, as_tuple=True)
        out = torch.zeros(layout.numel(), c["H"], dtype=torch.float64, device=DEV)
        out[rows[t, j].long()] = s["x"].double()[t]
        return (out, rows, layout, offsets) if c["to"] == "bf16" else (*_ratio64(out), rows, layout, offsets)
    if c["op"] == "int8":
        return (s["A"].double() * s["sa"].double()[:, None]) @ (s["B"].double() * s["sb"].double()[:, None]).T
    if c["op"] == "int8_grouped":
        out = torch.zeros(s["A"].shape[0], c["N"], dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            r = torch.nonzero(s["layout"] == e).flatten()
            out[r] = (s["A"][r].double() * s["sa"][r].double()[:, None]) @ \
                (s["B"][e].double() * s["sb"][e].double()[:, None]).T
        return out
    if c["op"] in ("combine", "combine_grad"):
        # by automatic differentiation of the weighted sum, in 64 bits
        t, j = torch.nonzero(s["rows"] >= 0, as_tuple=True)
        r = s["rows"][t, j].long()
        y, w = s["y"].double(), s["weights"].double()
        if c["op"] == "combine":
            return torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV).index_add_(0, t, y[r] * w[t, j][:, None])
        y.requires_grad_(True)
        w.requires_grad_(True)
        ((y[r] * w[t, j][:, None]) * s["grad"].double()[t]).sum().backward()
        return y.grad, w.grad
    z, I, some = s["z"].double(), c["I"], (s["layout"] >= 0).double()[:, None]
    if c["op"] == "gate":
        return _ratio64(z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:] * some)
    out = torch.zeros_like(z)
    for r0 in range(0, z.shape[0], 8192):
        part = z[r0:r0 + 8192].detach().requires_grad_(True)
        h = part[:, :I] * torch.sigmoid(part[:, :I]) * part[:, I:]
        (h * s["grad"][r0:r0 + 8192].double() * some[r0:r0 + 8192]).sum().backward()
        out[r0:r0 + 8192] = part.grad
    return out
