"""Measured cases of the operators around the FP8 products (include/dg_ops.h):
the expert router and its gradient, a whole mixture-of-experts layer for a few
tokens, and low-rank adapters of many requests beside a shared projection.

Every operator is given here in its plain form too: elementary torch
operations in 32 bits (64 where experts are ranked, so that borders between
neighbours do not depend on rounding), rounded once at the end.  ``run`` takes
the plain form or, with ``own``, the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-20  # added to the sum of a row's kept scores before dividing by it


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token through a 256-expert router: 8 groups, 4 kept, 8 experts
        dict(name="topk_token", op="topk", T=1, E=256, k=8, scoring="sigmoid", bias=True, n_group=8,
             topk_group=4, renorm=True, dtype="fp32", masked=0.0),
        # the same router over a prompt (the row count of the dense configurations)
        dict(name="topk_prompt", op="topk", T=4096, E=256, k=8, scoring="sigmoid", bias=True, n_group=8,
             topk_group=4, renorm=True, dtype="fp32", masked=0.0),
        # training step of a softmax router on bf16 logits
        dict(name="topk_grad_batch", op="topk_grad", T=8192, E=128, k=8, scoring="softmax", renorm=True,
             dtype="bf16", masked=0.0),
        # odd sizes: a ragged last micro-batch, some experts masked off
        dict(name="topk_grad_odd", op="topk_grad", T=333, E=61, k=5, scoring="sigmoid", renorm=True,
             dtype="fp32", masked=0.1),
        # one decoded token, eight experts of the two masked configurations' shapes
        dict(name="moe_token", op="moe", T=1, E=16, k=8, H=7168, I=2048, local=1.0, scales="fp32"),
        # a small layer, few tokens: bound by latency
        dict(name="moe_small", op="moe", T=3, E=5, k=2, H=640, I=384, local=1.0, scales="fp32"),
        # a decode batch in which every expert of this GPU has rows
        dict(name="moe_batch", op="moe", T=64, E=16, k=8, H=7168, I=2048, local=1.0, scales="fp32"),
        # the largest batch with experts spread over GPUs: most routed pairs are elsewhere
        dict(name="moe_spread", op="moe", T=251, E=16, k=8, H=7168, I=2048, local=0.125, scales="e8m0"),
        # one decoded token of one request beside the shared projection
        dict(name="lora_token", op="lora", M=1, N=7168, K=2048, R=16, L=4, rows="mixed", scales="fp32"),
        # a decode batch, every row its own adapter or none
        dict(name="lora_batch", op="lora", M=64, N=2112, K=7168, R=32, L=64, rows="each", scales="fp32"),
        # prompts of several requests packed into one call
        dict(name="lora_prompt", op="lora", M=4096, N=7168, K=2048, R=64, L=8, rows="runs", scales="fp32"),
        # odd sizes, rows of all adapters interleaved
        dict(name="lora_odd", op="lora", M=301, N=520, K=768, R=24, L=7, rows="mixed", scales="e8m0"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(("topk", "topk_grad", "moe", "moe", "lora", "lora"))
    if op in ("topk", "topk_grad"):
        n_group = rng.choice((1, 1, 2, 4, 8)) if op == "topk" else 1
        E = n_group * max(2, _log(rng, 8, 256) // n_group)
        topk_group = rng.randint((n_group + 1) // 2, n_group)
        k = rng.randint(1, min(8, E // n_group * topk_group))
        c = dict(op=op, T=_log(rng, 1, 4096), E=E, k=k, scoring=rng.choice(("softmax", "sigmoid")),
                 renorm=rng.random() < 0.7, dtype=rng.choice(("fp32", "bf16")),
                 masked=rng.choice((0.0, 0.05, 0.5 if E >= 32 else 0.0)))
        if op == "topk_grad" and c["renorm"]:
            c["k"] = max(2, k)  # one expert's weight is 1 whatever its logit: no gradient but noise
        if op == "topk":
            c.update(bias=rng.random() < 0.5, n_group=n_group, topk_group=topk_group)
        return c
    if op == "moe":
        T, E = _log(rng, 1, 256), rng.randint(2, 16)
        local = rng.choice((1.0, 0.5, 0.25)) if T <= 64 else rng.choice((0.25, 0.125))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), H=128 * _log(rng, 1, 56),
                    I=128 * _log(rng, 1, 16), local=local, scales=rng.choice(("fp32", "e8m0")))
    N, K = 8 * _log(rng, 16, 896), 128 * _log(rng, 1, 56)
    M = min(_log(rng, 1, 4096), 60_000_000_000 // (N * K))
    return dict(op=op, M=M, N=N, K=K, R=8 * _log(rng, 1, 16), L=_log(rng, 1, 64),
                rows=rng.choice(("mixed", "each", "runs")), scales=rng.choice(("fp32", "e8m0")))


# --------------------------------------------------------- inputs of the cases

def _e4m3(v):
    """e4m3 codes, as bytes, of values within +-448."""
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def _scale(amax, kind):
    """fp32 scale of blocks with these largest magnitudes, or the exponent e of 2^e."""
    if kind == "fp32":
        return amax / 448.0
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1): the least e' with amax <= 1.75 2^(e'+8)
    return torch.where(amax > 0, (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-127), torch.full_like(e, -127))


def _pad4(s):
    """Exponents as E8M0 bytes, rows padded to a multiple of four."""
    kb = s.shape[-1]
    out = torch.zeros(*s.shape[:-1], (kb + 3) // 4 * 4, dtype=torch.uint8, device=s.device)
    out[..., :kb] = (s + 127).to(torch.uint8)
    return out


def _divisor(s, kind):
    return s if kind == "fp32" else torch.ldexp(torch.ones_like(s, dtype=torch.float32), s)


def _tokens(x, kind):
    """Codes of x [..., K] with a scale per row and 128 columns."""
    b = x.float().unflatten(-1, (-1, 128))
    s = _scale(b.abs().amax(-1), kind)
    d = _divisor(s, kind).unsqueeze(-1)
    q = _e4m3(torch.where(d > 0, b / d, torch.zeros_like(b))).flatten(-2)
    return q, (s if kind == "fp32" else _pad4(s))


def _weights(gen, G, N, K, kind):
    """Codes of G random weights [N, K] with a scale per 128 x 128 block."""
    NB = (N + 127) // 128
    q = torch.empty(G, N, K, dtype=torch.uint8, device=DEV)
    s = []
    for g in range(G):
        w = torch.randn(N, K, generator=gen, device=DEV) * K ** -0.5
        p = torch.zeros(NB * 128, K, device=DEV)
        p[:N] = w
        b = p.view(NB, 128, K // 128, 128)
        e = _scale(b.abs().amax((1, 3)), kind)
        q[g] = _e4m3(b / _divisor(e, kind)[:, None, :, None]).view(NB * 128, K)[:N]
        s.append(e)
    s = torch.stack(s)
    return q, (s if kind == "fp32" else _pad4(s))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    randn = lambda *n: torch.randn(*n, generator=gen, device=DEV)  # noqa: E731
    c, s = dict(case), {"case": dict(case)}
    if c["op"] in ("topk", "topk_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        x = randn(T, E) * 1.5
        if c["masked"] > 0:  # experts that a row may not use; the first row may use none
            off = torch.rand(T, E, generator=gen, device=DEV) < c["masked"]
            off[0] = T > 1
            x = torch.where(off, torch.full_like(x, -math.inf), x)
        s["logits"] = x.to(torch.bfloat16) if c["dtype"] == "bf16" else x
        if c["op"] == "topk":
            s["bias"] = randn(E) * 0.1 if c["bias"] else None
        else:
            key = torch.where(x > -math.inf, x, torch.full_like(x, -math.inf))
            top = torch.sort(key, dim=1, descending=True, stable=True)
            s["ids"] = torch.where(top.values[:, :k] > -math.inf, top.indices[:, :k],
                                   torch.full((T, k), -1, device=DEV)).to(torch.int32).contiguous()
            s["grad"] = randn(T, k)
    elif c["op"] == "moe":
        T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
        s["x"], s["sx"] = _tokens(randn(T, H).to(torch.bfloat16), c["scales"])
        s["w13"], s["s13"] = _weights(gen, E, 2 * I, H, c["scales"])
        s["w2"], s["s2"] = _weights(gen, E, H, I, c["scales"])
        spread = max(E, int(round(E / c["local"])))  # experts of the whole layer; the first E are here
        ids = torch.rand(T, spread, generator=gen, device=DEV).argsort(1)[:, :k]
        s["ids"] = torch.where(ids < E, ids, torch.full_like(ids, -1)).to(torch.int32).contiguous()
        w = torch.exp(randn(T, k))
        s["weights"] = (w / w.sum(1, keepdim=True)).contiguous()
    else:
        M, N, K, R, L = (c[n] for n in ("M", "N", "K", "R", "L"))
        s["x"] = randn(M, K).to(torch.bfloat16)
        s["A"], s["sa"] = _tokens(s["x"], c["scales"])
        B, sb = _weights(gen, 1, N, K, c["scales"])
        s["B"], s["sb"] = B[0], sb[0].contiguous()
        s["lora_a"] = (randn(L, R, K) * K ** -0.5).to(torch.bfloat16)
        s["lora_b"] = (randn(L, N, R) * 0.3 * R ** -0.5).to(torch.bfloat16)
        s["scaling"] = 0.5 + torch.rand(L, generator=gen, device=DEV)
        if c["rows"] == "each":  # a decode batch: one row a request, the adapters in turn, every ninth row without
            ids = torch.arange(M, device=DEV) % L
            ids = torch.where(torch.arange(M, device=DEV) % 9 == 8, torch.full_like(ids, -1), ids)
        elif c["rows"] == "runs":  # packed prompts: runs of rows of uneven length
            cuts = torch.rand(M, generator=gen, device=DEV) < 1.0 / 300
            run_ids = torch.randint(-1, L, (M + 1,), generator=gen, device=DEV)
            ids = run_ids[torch.cumsum(cuts, 0)]
        else:
            ids = torch.randint(-1, L, (M,), generator=gen, device=DEV)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["D"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    return s


def work(case):
    c = case
    if c["op"] in ("topk", "topk_grad"):
        T, E, k, b = c["T"], c["E"], c["k"], 2 if c["dtype"] == "bf16" else 4
        if c["op"] == "topk":
            return {"bytes": T * E * b + T * k * 8 + (4 * E if c["bias"] else 0), "flops": 4 * T * E}
        return {"bytes": 2 * T * E * b + T * k * 8, "flops": 4 * T * E}
    scale = 4 if c["scales"] == "fp32" else 1
    if c["op"] == "moe":
        T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
        spread = max(E, int(round(E / c["local"])))
        pairs = T * k * E / spread
        active = E * (1.0 - (1.0 - k / spread) ** T)  # experts with a row, on average
        return {"bytes": int(active * 3 * H * I * (1 + scale / 16384) + T * H * (1 + scale / 128) + T * H * 2 + T * k * 8),
                "flops": int(pairs * 6 * H * I)}
    M, N, K, R, L = (c[n] for n in ("M", "N", "K", "R", "L"))
    used = min(L, M)
    return {"bytes": int(M * K * (3 + scale / 128) + N * K * (1 + scale / 16384) + M * N * 2 + used * R * (K + N) * 2 + M * 4),
            "flops": 2 * M * N * K + 2 * M * R * (K + N)}


# ------------------------------------------------------------- the plain forms

def _topk_plain(x, bias, c):
    T, E, k, G = x.shape[0], c["E"], c["k"], c["n_group"]
    x = x.float()
    ok = x > -math.inf
    low = torch.full_like(x, -math.inf)
    xm = torch.where(ok, x, low)
    if bias is None and G == 1:
        rank = xm.double()
    else:
        xd = xm.double()
        if c["scoring"] == "sigmoid":
            rank = 1.0 / (1.0 + torch.exp(-xd))
        else:
            e = torch.where(ok, torch.exp(xd - xd.amax(1, keepdim=True)), torch.zeros_like(xd))
            rank = e / e.sum(1, keepdim=True)
        if bias is not None:
            rank = rank + bias.double()
        rank = torch.where(ok, rank, low.double())
    if G > 1:
        two = torch.sort(rank.view(T, G, E // G), dim=2, descending=True).values[:, :, :2]
        second = two[:, :, 1:].sum(2)  # a group with one open expert is ranked by that one
        total = two[:, :, 0] + torch.where(second > -math.inf, second, torch.zeros_like(second))
        best = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, best, True)
        rank = torch.where(keep.repeat_interleave(E // G, 1), rank, torch.full_like(rank, -math.inf))
    top = torch.sort(rank, dim=1, descending=True, stable=True)
    got = top.values[:, :k] > -math.inf
    at = top.indices[:, :k]
    if c["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-xm))
    else:
        e = torch.where(ok, torch.exp(xm - xm.amax(1, keepdim=True)), torch.zeros_like(xm))
        score = e / e.sum(1, keepdim=True)
    w = torch.where(got, score.gather(1, at), torch.zeros(T, k, device=x.device))
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + EPS)
    return torch.where(got, at, torch.full_like(at, -1)).to(torch.int32), w


def _topk_grad_plain(s, c):
    x = s["logits"].float()
    T, E = x.shape
    ok = x > -math.inf
    if c["scoring"] == "sigmoid":
        score = torch.where(ok, 1.0 / (1.0 + torch.exp(-x)), torch.zeros_like(x))
    else:
        e = torch.where(ok, torch.exp(x - torch.where(ok, x, torch.full_like(x, -math.inf)).amax(1, keepdim=True)),
                        torch.zeros_like(x))
        score = torch.where(ok, e / e.sum(1, keepdim=True), torch.zeros_like(x))
    got = s["ids"] >= 0
    at = s["ids"].long().clamp(min=0)
    picked = torch.where(got, score.gather(1, at), torch.zeros_like(s["grad"]))
    g = torch.where(got, s["grad"], torch.zeros_like(s["grad"]))
    if c["renorm"]:
        total = picked.sum(1, keepdim=True) + EPS
        g = torch.where(got, (g - (g * picked).sum(1, keepdim=True) / total) / total, torch.zeros_like(g))
    full = torch.zeros(T, E, device=x.device).scatter_add_(1, at, g)  # gradient of the scores
    if c["scoring"] == "sigmoid":
        out = full * score * (1.0 - score)
    else:
        out = score * (full - (full * score).sum(1, keepdim=True))
    return out.to(s["logits"].dtype)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _per_row(s, kb, kind):
    return s if kind == "fp32" else torch.ldexp(torch.ones(s.shape[:-1] + (kb,), device=s.device), s[..., :kb].int() - 127)


def _rows_plain(q, s, kind):
    kb = q.shape[-1] // 128
    return (_values(q).unflatten(-1, (kb, 128)) * _per_row(s, kb, kind).unsqueeze(-1)).flatten(-2)


def _weights_plain(q, s, kind):
    N, kb = q.shape[-2], q.shape[-1] // 128
    s = _per_row(s, kb, kind).repeat_interleave(128, -2)[..., :N, :]
    return (_values(q).unflatten(-1, (kb, 128)) * s.unsqueeze(-1)).flatten(-2)


def _moe_plain(s, c):
    I, E, kind = c["I"], c["E"], c["scales"]
    x = _rows_plain(s["x"], s["sx"], kind)
    both = torch.matmul(x.unsqueeze(0), _weights_plain(s["w13"], s["s13"], kind).transpose(1, 2))
    gate, up = both[..., :I], both[..., I:]
    hq, hs = _tokens(gate / (1.0 + torch.exp(-gate)) * up, kind)
    out = torch.matmul(_rows_plain(hq, hs, kind), _weights_plain(s["w2"], s["s2"], kind).transpose(1, 2))
    here = s["ids"].unsqueeze(0) == torch.arange(E, device=x.device).view(E, 1, 1)
    w = (here * s["weights"].unsqueeze(0)).sum(2)
    return (out * w.unsqueeze(2)).sum(0).to(torch.bfloat16)


def _lora_plain(s, c):
    L, R, kind = c["L"], c["R"], c["scales"]
    base = torch.matmul(_rows_plain(s["A"], s["sa"], kind), _weights_plain(s["B"], s["sb"], kind).T)
    low = torch.matmul(s["x"].float(), s["lora_a"].float().flatten(0, 1).T).view(-1, L, R)
    mine = s["ids"].view(-1, 1) == torch.arange(L, device=low.device)
    low = low * (mine * s["scaling"]).unsqueeze(2)
    return (base + torch.matmul(low.flatten(1), s["lora_b"].float().transpose(1, 2).flatten(0, 1))).to(torch.bfloat16)


def run(state):
    c, s = state["case"], state
    if not own:
        if c["op"] == "topk":
            return _topk_plain(s["logits"], s["bias"], c)
        return {"topk_grad": _topk_grad_plain, "moe": _moe_plain, "lora": _lora_plain}[c["op"]](s, c)
    import fp8_block_scaled_gemm_amd as dg
    if c["op"] == "topk":
        return dg.dg_moe_topk(s["logits"], c["k"], bias=s["bias"], n_group=c["n_group"],
                              topk_group=c["topk_group"], scoring=c["scoring"], renormalize=c["renorm"])
    if c["op"] == "topk_grad":
        return dg.dg_moe_topk_backward(s["logits"], s["ids"], s["grad"], scoring=c["scoring"],
                                       renormalize=c["renorm"])
    if c["op"] == "moe":
        call = dg.dg_moe_mlp_fp8 if c["scales"] == "fp32" else dg.dg_moe_mlp_fp8_e8m0
        return call(s["x"], s["sx"], s["ids"], s["weights"], s["w13"], s["s13"], s["w2"], s["s2"])
    call = dg.dg_fp8_gemm_nt_lora if c["scales"] == "fp32" else dg.dg_fp8_gemm_nt_lora_e8m0
    return call(s["A"], s["sa"], s["B"], s["sb"], s["D"], s["x"], s["lora_a"], s["lora_b"], s["ids"], s["scaling"])


# ------------------------------------------------------ the definition, 64 bits

def _grid8(v):
    """Nearest e4m3 value of doubles within +-448, ties to even."""
    e = torch.floor(torch.log2(torch.where(v == 0, torch.ones_like(v), v.abs()))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _code64(q):
    b = q.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (1.0 + m / 8) * torch.exp2((e - 7).double()), m * 2.0 ** -9)
    return torch.where(b >= 128, -mag, mag)


def _scale64(s, kind):
    return s.double() if kind == "fp32" else torch.exp2(s.double() - 127)


def _row64(q, s, kind):
    """One [rows, K] operand with a scale per row and 128 columns."""
    v = _code64(q).view(q.shape[0], -1, 128)
    return (v * _scale64(s, kind)[:, :v.shape[1], None]).reshape(q.shape[0], -1)


def _block64(q, s, kind):
    N, K = q.shape
    row = torch.arange(N, device=q.device) // 128
    col = torch.arange(K, device=q.device) // 128
    return _code64(q) * _scale64(s, kind)[row][:, col]


def _log_sum(x):
    top = np.maximum(x.max(1, keepdims=True), -1e300)
    return top + np.log(np.maximum(np.exp(x - top).sum(1, keepdims=True), 1e-300))


def _picked64(x, p, bias, c):
    """The scores of one row's experts, best first: an ordinary loop over the definition."""
    rank = x if bias is None and c["n_group"] == 1 else p if bias is None else p + bias
    rank = [r if x[e] > -math.inf else -math.inf for e, r in enumerate(rank)]
    size = c["E"] // c["n_group"]
    pair = [[r for r in sorted(rank[g * size:(g + 1) * size])[-2:] if r > -math.inf] for g in range(c["n_group"])]
    groups = sorted(range(c["n_group"]), key=lambda g: (-sum(pair[g]) if pair[g] else math.inf, g))
    open_to = [e for g in groups[:c["topk_group"]] for e in range(g * size, (g + 1) * size) if rank[e] > -math.inf]
    best = sorted(open_to, key=lambda e: (-rank[e], e))[:c["k"]]
    return [p[e] for e in best] + [0.0] * (c["k"] - len(best))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "topk":
        x = s["logits"].double().cpu().numpy()
        p = 1 / (1 + np.exp(-x)) if c["scoring"] == "sigmoid" else np.exp(x - _log_sum(x))
        bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
        w = torch.zeros(x.shape[0], c["k"], dtype=torch.float64)
        for t in range(x.shape[0]):
            w[t, :] = torch.tensor(_picked64(x[t], p[t], bias, c))
        w = w.to(DEV)
        return None, (w / (w.sum(1, keepdim=True) + EPS) if c["renorm"] else w)
    if c["op"] == "topk_grad":
        # by automatic differentiation of the weights, in 64 bits
        x = s["logits"].double().nan_to_num(neginf=-1e300).requires_grad_(True)
        some = s["ids"] >= 0
        p = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, 1)
        w = p.gather(1, s["ids"].long().clamp(min=0)) * some
        if c["renorm"]:
            w = w / (w.sum(1, keepdim=True) + EPS)
        (w * s["grad"].double() * some).sum().backward()
        return torch.where(s["logits"] > -math.inf, x.grad, torch.zeros_like(x))
    kind = c["scales"]
    if c["op"] == "moe":
        x = _row64(s["x"], s["sx"], kind)
        y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            if t.numel() == 0:
                continue
            z = x[t] @ _block64(s["w13"][e], s["s13"][e], kind).T
            h = (z[:, :c["I"]] * torch.sigmoid(z[:, :c["I"]]) * z[:, c["I"]:]).view(t.numel(), -1, 128)
            top = h.abs().amax(2, keepdim=True)
            if kind == "fp32":
                d = top / 448
            else:
                d = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 448)).clamp(min=-127))
            h = torch.where(top > 0, _grid8(h / torch.where(top > 0, d, torch.ones_like(d))) * d, torch.zeros_like(h))
            out = h.view(t.numel(), -1) @ _block64(s["w2"][e], s["s2"][e], kind).T
            y.index_add_(0, t, out * s["weights"][t, j].double().unsqueeze(1))
        return y
    out = _row64(s["A"], s["sa"], kind) @ _block64(s["B"], s["sb"], kind).T
    for a in range(c["L"]):
        t = torch.nonzero(s["ids"] == a).flatten()
        if t.numel():
            low = (s["x"][t].double() @ s["lora_a"][a].double().T) * s["scaling"][a].double()
            out[t] += low @ s["lora_b"][a].double().T
    return out
