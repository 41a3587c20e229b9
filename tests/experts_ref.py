"""Plain implementations of include/dg_experts.h and include/dg_int8.h in 64
bits, from their definitions with numpy, and bounds on a kernel's error.

Bounds count roundings: half a step, eps/2 relative, of each type (bf16 2^-8,
fp32 2^-24, e4m3 2^-4)."""
from __future__ import annotations

import numpy as np

from tests.ops_ref import BF16, FP32, e4m3_step, e4m3_value

BF16_TINY = 2.0 ** -134  # half a step of the smallest bf16
SILU_TINY = 1.05e-36     # see swiglu


def bf16_error(v):
    return BF16 * np.abs(v) + BF16_TINY


# -------------------------------------------------------------------- sorting

def sort_rows(T, k, E):
    P = T * k
    return (P + 127 * min(E, P)) // 128 * 128


def sort(ids, E, M):
    """(rows, layout, offsets) by an ordinary loop."""
    mine = [[] for _ in range(E)]
    for p, e in enumerate(ids.ravel().tolist()):
        if 0 <= e < E:
            mine[e].append(p)
    rows, layout, offsets = np.full(ids.size, -1, np.int32), np.full(M, -1, np.int32), [0]
    for e, pairs in enumerate(mine):
        for i, p in enumerate(pairs):
            rows[p], layout[offsets[-1] + i] = offsets[-1] + i, e
        offsets.append(offsets[-1] + -(-len(pairs) // 128) * 128)
    return rows.reshape(ids.shape), layout, np.array(offsets, np.int32)


# --------------------------------------------------------------- weighted sum

def unpermute(y, rows, weights):
    """(out, bound): fp32 sums in the order of the choices, rounded to bf16."""
    T, k = rows.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= rows[t, j] < y.shape[0]:
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * y[rows[t, j]]
                mag[t] += np.abs(w * y[rows[t, j]])
    tol = k * FP32 * mag
    return out, tol + bf16_error(np.abs(out) + tol)


def unpermute_backward(g, y, rows, weights):
    """(grad_y, bound, grad_weights, bound); rows that no pair names are zeros."""
    T, k = rows.shape
    H = g.shape[1]
    gy, gw, mag = np.zeros_like(y), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = rows[t, j]
            if 0 <= r < y.shape[0]:
                gy[r] = (1.0 if weights is None else float(weights[t, j])) * g[t]
                gw[t, j], mag[t, j] = g[t] @ y[r], np.abs(g[t]) @ np.abs(y[r])
    chain = 8 * (H // 2048 + 1) + 9  # a thread's products, six steps over a wave, three over the waves
    return gy, bf16_error(gy) + 2 * FP32 * np.abs(gy), gw, chain * FP32 * mag


# ------------------------------------------------------------------- the gate

def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g))


def swiglu(z):
    """(h, bound on fp32 arithmetic): the exponential's own error, a sum, a
    quotient and a product, each a rounding or two.  A sigmoid below the smallest
    normal fp32, 2^-126, may come as 0: there the gate is below -87.3, and where it
    is below -88.8 silu itself is smaller than what that gives, so that the error
    is at most 88.8 * 2^-126 = 1.05e-36 times |up|."""
    I = z.shape[1] // 2
    g, u = z[:, :I], z[:, I:]
    h = g * sigmoid(g) * u
    return h, 8 * FP32 * np.abs(h) + SILU_TINY * np.abs(u) + 2.0 ** -149


def swiglu_backward(z, d):
    """(grad_z, bound): 1 - p is off by the sigmoid's error, times the gate."""
    I = z.shape[1] // 2
    g, u, p = z[:, :I], z[:, I:], sigmoid(z[:, :I])
    out = np.concatenate((d * u * p * (1 + g * (1 - p)), d * g * p), 1)
    off = np.concatenate((np.abs(d * u) * (p * (8 * np.abs(g) + 16) * FP32 + 1e-35),
                          np.abs(d) * (12 * FP32 * np.abs(g * p) + SILU_TINY)), 1) + 2.0 ** -149
    return out, off + bf16_error(np.abs(out) + off)


# -------------------------------------------------------------------- quantized

def check_fp8(q, s, v, err):
    """Codes q [M][W] uint8 with fp32 scales [M][W/128] against values v that
    are known to err: the scale is amax / 448, a code is the nearest e4m3."""
    b, e = v.reshape(v.shape[0], -1, 128), err.reshape(v.shape[0], -1, 128)
    top, dt = np.abs(b).max(2), e.max(2)
    s = s.astype(np.float64)
    assert (np.abs(s - top / 448) <= dt / 448 + FP32 * top / 448 + 2.0 ** -149).all()
    got = e4m3_value(q).reshape(b.shape) * s[:, :, None]
    slack = e + (dt[:, :, None] / np.where(top > 0, top, 1)[:, :, None] + 4 * FP32) * np.abs(b)
    safe = np.where(s > 0, s, 1.0)[:, :, None]
    half = e4m3_step(np.minimum((np.abs(b) + slack) / safe, 448)) / 2
    assert (np.abs(got - b) <= np.where(s[:, :, None] > 0, half * safe, np.abs(b)) + slack).all()


def quantize_int8(x):
    """(codes, scales) of fp32 rows, by the recipe itself in fp32."""
    x = x.astype(np.float32)
    s = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)
    safe = np.where(s > 0, s, np.float32(1))[:, None]
    q = np.clip(np.rint((x / safe).astype(np.float32)), -127, 127)
    return np.where(s[:, None] > 0, q, 0).astype(np.int8), s


def check_int8(q, s, v, err):
    top, dt = np.abs(v).max(1), err.max(1)
    s = s.astype(np.float64)
    assert (np.abs(s - top / 127) <= dt / 127 + FP32 * top / 127 + 2.0 ** -149).all()
    slack = err + (dt / np.where(top > 0, top, 1) + 4 * FP32)[:, None] * np.abs(v)
    assert (np.abs(q * s[:, None] - v) <= s[:, None] / 2 + slack).all()


def int8_product(A, sa, B, sb):
    """fp32 as the definition rounds it: (sa sb) times the exact sum's fp32."""
    sums = A.astype(np.int64) @ B.astype(np.int64).T
    assert np.abs(sums).max(initial=0) < 2 ** 31
    with np.errstate(over="ignore", invalid="ignore"):
        return (sa.astype(np.float32)[:, None] * sb.astype(np.float32)) * sums.astype(np.float32)
