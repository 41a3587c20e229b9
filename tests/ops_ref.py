"""Plain 64-bit implementations of the operators of include/dg_ops.h, written
from their definitions with numpy, and the error bounds their tests use.

Bounds count the roundings the kernels make: half a step, eps/2 relative, of
each type (bf16 2^-8, fp32 2^-24, e4m3 2^-4), times the magnitude the rounded
value enters with.  FP8 products are accumulated by the matrix unit, whose
internal alignment is not documented: their error is bounded by PRODUCT times
the sum of the absolute products."""
from __future__ import annotations

import math

import numpy as np

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
PRODUCT = 2.0 ** -16
EPS = 1e-20


# ---------------------------------------------------------------- formats

def e4m3_value(codes: np.ndarray) -> np.ndarray:
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * np.exp2((e - 7).astype(np.float64)), m * 2.0 ** -9)
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c >= 128, -v, v)


def e4m3_step(v: np.ndarray) -> np.ndarray:
    """Distance between the e4m3 values around |v|."""
    a = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    return np.exp2(np.where(a > 0, e, -6.0) - 3)


def e4m3_round(v: np.ndarray) -> np.ndarray:
    s = e4m3_step(v)
    return np.clip(np.round(v / s) * s, -448, 448)


def block_scale(amax: np.ndarray, kind: str) -> np.ndarray:
    if kind == "fp32":
        return (amax.astype(np.float32) / np.float32(448)).astype(np.float64)
    e = np.ceil(np.log2(np.maximum(amax, 2.0 ** -300) / 448))
    e = np.where(amax <= 448 * np.exp2(e - 1), e - 1, e)  # log2 may round up over a border
    return np.exp2(np.maximum(e, -127))


def scale_values(s: np.ndarray, kb: int, kind: str) -> np.ndarray:
    s = s[..., :kb].astype(np.float64)
    return s if kind == "fp32" else np.exp2(s - 127)


def rows_value(q, s, kind):
    kb = q.shape[-1] // 128
    v = e4m3_value(q).reshape(q.shape[0], kb, 128) * scale_values(s, kb, kind)[:, :, None]
    return v.reshape(q.shape)


def block_value(q, s, kind):
    n, k = q.shape
    s = scale_values(s, k // 128, kind)
    return e4m3_value(q) * s[np.arange(n) // 128][:, np.arange(k) // 128]


# ----------------------------------------------------------------- inputs

def quantize_rows(x: np.ndarray, kind: str):
    kb = x.shape[1] // 128
    b = x.astype(np.float64).reshape(x.shape[0], kb, 128)
    s = block_scale(np.abs(b).max(2), kind)
    return _encode(np.where(s[:, :, None] > 0, b / np.where(s > 0, s, 1)[:, :, None], 0.0).reshape(x.shape)), \
        _scale_array(s, kind)


def quantize_blocks(w: np.ndarray, kind: str):
    n, k = w.shape
    nb, kb = (n + 127) // 128, k // 128
    s = np.zeros((nb, kb))
    for i in range(nb):
        for j in range(kb):
            s[i, j] = block_scale(np.abs(w[128 * i:128 * i + 128, 128 * j:128 * j + 128]).max(), kind)
    return _encode(w / s[np.arange(n) // 128][:, np.arange(k) // 128]), _scale_array(s, kind)


def _encode(v):
    v = e4m3_round(v)
    a = np.abs(v)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    normal = a >= 2.0 ** -6
    m = np.where(normal, np.round((a / np.exp2(e) - 1) * 8), np.round(a * 2.0 ** 9)).astype(np.int64)
    code = np.where(normal, ((e + 7).astype(np.int64) << 3) | m, m)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _scale_array(s, kind):
    if kind == "fp32":
        return s.astype(np.float32)
    out = np.zeros(s.shape[:-1] + ((s.shape[-1] + 3) // 4 * 4,), np.uint8)
    out[..., :s.shape[-1]] = (np.log2(s) + 127).astype(np.uint8)
    return out


# ----------------------------------------------------------------- router

def _scores(x, scoring):
    """p of one row in 64 bits; masked logits (NaN, -inf) count nothing."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-x))
    top = x.max()
    if top == -np.inf:
        return np.zeros_like(x)
    e = (x == np.inf).astype(np.float64) if top == np.inf else np.exp(x - top)
    return e / e.sum()


def topk(x, bias, k, n_group, topk_group, scoring, renorm, scale):
    T, E = x.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    size = E // n_group
    for t in range(T):
        p = _scores(x[t], scoring)
        rank = x[t].astype(np.float64) if bias is None and n_group == 1 else \
            p + (0 if bias is None else bias.astype(np.float64))
        is_open = (x[t] > -np.inf) & (rank > -np.inf)
        if n_group > 1:
            value = []
            for g in range(n_group):
                r = sorted((rank[e] for e in range(g * size, (g + 1) * size) if is_open[e]), reverse=True)
                value.append(sum(r[:2]) if r else -math.inf)
            kept = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
            is_open &= np.isin(np.arange(E) // size, kept)
        best = sorted((e for e in range(E) if is_open[e]), key=lambda e: (-rank[e], e))[:k]
        ids[t, :len(best)] = best
        w[t, :len(best)] = p[best]
        if renorm:
            w[t] /= w[t].sum() + EPS
    return ids, w * scale


def topk_weights(x, ids, scoring, renorm, scale):
    """Weights as a function of the logits, the experts fixed."""
    w = np.zeros(ids.shape)
    for t in range(x.shape[0]):
        p = _scores(x[t], scoring)
        for j, e in enumerate(ids[t]):
            w[t, j] = p[e] if 0 <= e < x.shape[1] else 0.0
        if renorm:
            w[t] /= w[t].sum() + EPS
    return w * scale


def topk_backward(x, ids, gw, scoring, renorm, scale):
    """(gradient, magnitude of the terms it is the sum of)."""
    T, E = x.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        p = _scores(x[t], scoring)
        at = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < E]
        g, ga = np.zeros(E), np.zeros(E)
        S = sum(p[e] for _, e in at) + EPS
        mean = sum(gw[t, j] * scale * p[e] for j, e in at) / S
        mean_a = sum(abs(gw[t, j] * scale) * p[e] for j, e in at) / S
        for j, e in at:
            v = float(gw[t, j]) * scale
            g[e] += (v - mean) / S if renorm else v
            ga[e] += (abs(v) + mean_a) / S if renorm else abs(v)
        if scoring == "sigmoid":
            out[t], mag[t] = g * p * (1 - p), ga * p * (1 - p) + ga * p * FP32
        else:
            out[t], mag[t] = p * (g - (g * p).sum()), p * (ga + (ga * p).sum())
    return out, mag


# ------------------------------------------------------------ expert layer

def moe(x, sx, ids, weights, w13, s13, w2, s2, kind):
    """(y, bound on a kernel's error before the rounding to bf16)."""
    T, H = x.shape
    E, _, I = w2.shape
    xv = rows_value(x, sx, kind)
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        pairs = [(t, j) for t in range(T) for j in range(ids.shape[1]) if ids[t, j] == e]
        if not pairs:
            continue
        t = np.array([p[0] for p in pairs])
        a, b = block_value(w13[e], s13[e], kind), block_value(w2[e], s2[e], kind)
        z, dz = xv[t] @ a.T, (np.abs(xv[t]) @ np.abs(a).T) * PRODUCT
        g, u, dg, du = z[:, :I], z[:, I:], dz[:, :I], dz[:, I:]
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        h = silu * u
        # |silu'| <= 1.1; a few fp32 roundings and the exponential's own
        dh = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 16 * FP32 * (1 + np.abs(g)) * np.abs(h)
        hb, db = h.reshape(len(t), I // 128, 128), dh.reshape(len(t), I // 128, 128)
        amax = np.abs(hb).max(2, keepdims=True)
        d = block_scale(amax, kind)
        safe = np.where(d > 0, d, 1.0)
        q = np.where(d > 0, e4m3_round(hb / safe), 0.0)
        # a value within its error of a rounding border may take either code
        at_max = db.max(2, keepdims=True) / safe / 448 + 4 * FP32
        slack = db / safe + np.abs(hb / safe) * (at_max if kind == "fp32" else 0.0)
        other = np.maximum(np.abs(e4m3_round(hb / safe + slack) - q), np.abs(e4m3_round(hb / safe - slack) - q))
        off = np.where(d > 0, other * d + (np.abs(q) * d * at_max if kind == "fp32" else 0.0), db)
        if kind == "e8m0":  # so may the block's power of two: then every code is rounded anew
            edge = np.abs(np.log2(np.where(amax > 0, amax, 1.0) / 448) % 1.0)
            near = np.minimum(edge, 1 - edge) < 4 * at_max  # d >= amax / 448, at most twice that
            off = np.where(near, np.abs(hb) * 2.0 ** -3 + d * 2.0 ** -9, off)
        hv, off = (q * d).reshape(len(t), I), off.reshape(len(t), I)
        wt = np.array([float(weights[p]) for p in pairs])[:, None]
        o = hv @ b.T
        np.add.at(y, t, wt * o)
        np.add.at(tol, t, np.abs(wt) * (off @ np.abs(b).T + (np.abs(hv) @ np.abs(b).T) * PRODUCT * 2))
    return y, tol


# --------------------------------------------------------- low-rank adapters

def lora(A, sa, B, sb, x, la, lb, ids, scaling, kind):
    """(D, bound on a kernel's error before the rounding to bf16)."""
    a, b = rows_value(A, sa, kind), block_value(B, sb, kind)
    out, tol = a @ b.T, (np.abs(a) @ np.abs(b).T) * PRODUCT
    for m, i in enumerate(ids):
        if 0 <= i < la.shape[0]:
            v, va = x[m] @ la[i].T * scaling[i], np.abs(x[m]) @ np.abs(la[i]).T * abs(scaling[i])
            out[m] += v @ lb[i].T
            # two bf16 parts leave 2^-17 of the vector; fp32 sums over K and R
            tol[m] += (va * PRODUCT) @ np.abs(lb[i]).T * 2
    return out, tol
