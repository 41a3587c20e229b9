"""The steps of an expert layer for many tokens (include/dg_experts.h) on the
GPU against their definitions, at the sizes and choices where they can go wrong."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import experts_ref as ref
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def choices(rng, T, k, E, kind):
    if kind == "own":  # different experts in a row
        return np.stack([rng.permutation(max(E, k))[:k] for _ in range(T)]).astype(np.int32).reshape(T, k) if T else \
            np.zeros((0, k), np.int32)
    if kind == "any":  # repeated ones, and some elsewhere
        return rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    if kind == "one":
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    ids = rng.integers(0, E, (T, k)).astype(np.int64)  # far outside
    ids[rng.random((T, k)) < 0.3] = 2 ** 31 - 1
    ids[rng.random((T, k)) < 0.3] = -2 ** 31
    return ids.astype(np.int32)


SORTS = [  # T, k, E, kind
    (1, 8, 256, "own"), (1, 1, 1, "own"), (3, 2, 5, "any"), (0, 4, 7, "own"), (40, 64, 3, "any"), (200, 5, 61, "far"),
    (333, 5, 31, "any"), (128, 1, 1, "one"), (129, 1, 2, "one"), (64, 8, 4096, "own"), (700, 3, 9, "none"),
    (1024, 8, 16, "any"), (1025, 8, 256, "own"), (4096, 8, 256, "own"), (4097, 3, 4096, "any"), (9000, 1, 7, "one"),
    (8193, 2, 300, "far"), (30000, 10, 64, "any"),
]


@pytest.mark.parametrize("T,k,E,kind", SORTS)
def test_sort_matches_definition(T, k, E, kind):
    ids = choices(np.random.default_rng(T + E), T, k, E, kind)
    M = dg.dg_moe_sort_rows(T, k, E)
    assert M == ref.sort_rows(T, k, E)
    want = ref.sort(ids, E, M)
    for got, w in zip(dg.dg_moe_sort(to_dev(ids), E), want):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), w)


def test_sort_into_larger_buffers_that_held_other_values():
    ids = choices(np.random.default_rng(4), 70, 6, 20, "any")
    M = dg.dg_moe_sort_rows(70, 6, 20) + 384
    full = lambda *n: torch.full(n, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    rows, layout, offsets = full(70, 6), full(M), full(21)
    got = dg.dg_moe_sort(to_dev(ids), 20, rows, layout, offsets)
    assert got[0] is rows and got[1] is layout and got[2] is offsets
    for g, w in zip(got, ref.sort(ids, 20, M)):
        assert np.array_equal(g.cpu().numpy(), w)


# ------------------------------------------------------------------ dispatch

DISPATCHES = [  # T, k, E, kind, H
    (1, 8, 256, "own", 7168), (0, 3, 5, "own", 256), (5, 2, 4, "any", 128), (37, 3, 6, "any", 384), (333, 5, 31, "far", 640),
    (61, 20, 7, "any", 1152), (1030, 8, 40, "own", 256), (9, 1, 3, "none", 128),
    (3, 2, 5, "any", 8320), (130, 33, 6, "any", 8320),
]


def plan_of(ids, E):
    M = dg.dg_moe_sort_rows(ids.shape[0], ids.shape[1], E)
    return ref.sort(ids, E, M)


def check_plan(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("T,k,E,kind,H", DISPATCHES + [(50, 4, 9, "any", 8), (77, 3, 12, "any", 1416)])
def test_dispatch_copies_rows_and_clears_padding(T, k, E, kind, H):
    rng = np.random.default_rng(T + H)
    ids = choices(rng, T, k, E, kind)
    x = bf16(rng.standard_normal((T, H)))
    want = plan_of(ids, E)
    given = torch.full((want[1].size, H), 5.0, dtype=torch.bfloat16, device="cuda")
    for out in (None, given):
        got = dg.dg_moe_dispatch(x, to_dev(ids), E, out)
        check_plan(got[1:], want)
        full = np.zeros((want[1].size, H))
        some = want[0] >= 0
        full[want[0][some]] = host(x)[np.nonzero(some)[0]]
        assert np.array_equal(host(got[0]), full)
    assert got[0] is given


@pytest.mark.parametrize("kind_of", ["fp8", "e8m0", "int8"])
@pytest.mark.parametrize("T,k,E,kind,H", DISPATCHES)
def test_dispatch_quantizes_like_the_token_quantizers(T, k, E, kind, H, kind_of):
    rng = np.random.default_rng(T + H)
    ids = choices(rng, T, k, E, kind)
    x = bf16(rng.standard_normal((T, H)) * np.exp(rng.standard_normal((T, 1)) * 4))
    if T > 2:
        x[1] = 0
        x[2, :128] = 0
        x[0, :100] = 1e-40  # subnormal
    want = plan_of(ids, E)
    M = want[1].size
    call = {"fp8": dg.dg_moe_dispatch_fp8, "e8m0": dg.dg_moe_dispatch_fp8_e8m0, "int8": dg.dg_moe_dispatch_int8}[kind_of]
    if kind_of == "int8":
        q = torch.full((M, H), 99, dtype=torch.int8, device="cuda")
        s = torch.full((M,), 9.0, device="cuda")
        cq, cs = (to_dev(a) for a in ref.quantize_int8(x.float().cpu().numpy())) if T else (q[:0], s[:0])
    else:
        q = torch.full((M, H), 99, dtype=torch.uint8, device="cuda")
        if kind_of == "fp8":
            s = torch.full((M, H // 128), 9.0, device="cuda")
            cq, cs = dg.dg_quantize_fp8_per_token_bf16(x)
        else:
            s = torch.full((M, dg.e8m0_pitch(H // 128)), 9, dtype=torch.uint8, device="cuda")
            cs = torch.full((T, dg.e8m0_pitch(H // 128)), 9, dtype=torch.uint8, device="cuda")
            cq, cs = dg.dg_quantize_fp8_per_token_e8m0(x.float(), None, cs)
    got = call(x, to_dev(ids), E, q, s)
    assert got[0] is q and got[1] is s
    check_plan(got[2:], want)
    wq, ws = q.clone().fill_(99), s.clone().fill_(9)
    t, j = np.nonzero(want[0] >= 0)
    at, t = torch.from_numpy(want[0][t, j].astype(np.int64)).cuda(), torch.from_numpy(t).cuda()
    wq[at], ws[at] = cq[t], cs[t]
    zero = (wq & 0x7F) == 0 if kind_of != "int8" else wq == 200  # +0 and -0 count as one
    assert torch.equal(torch.where(zero, wq & 0x7F, wq), torch.where(zero, q & 0x7F, q)) and torch.equal(s, ws)
    if T:  # and into new buffers
        new = call(x, to_dev(ids), E)
        held = H // 128 if kind_of == "e8m0" else None  # without the scales' padding bytes
        assert torch.equal(new[0][at], q[at]) and torch.equal(new[1][at][..., :held], s[at][..., :held])
        assert new[0].shape == q.shape and new[1].shape == s.shape


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_dispatch_marks_blocks_that_are_not_finite(bad):
    x = torch.randn(3, 384, device="cuda").to(torch.bfloat16)
    x[1, 130] = bad
    ids = torch.tensor([[0], [1], [1]], dtype=torch.int32, device="cuda")
    q, s, rows, _, _ = dg.dg_moe_dispatch_fp8(x, ids, 2)
    assert torch.equal(torch.isnan(s[rows[:, 0].long()]),
                       torch.tensor([[False] * 3, [False, True, False], [False] * 3], device="cuda"))
    q, s, rows, _, _ = dg.dg_moe_dispatch_fp8_e8m0(x, ids, 2)
    assert (s[rows[:, 0].long()] == 255).nonzero().tolist() == [[1, 1]]
    q, s, rows, _, _ = dg.dg_moe_dispatch_int8(x, ids, 2)
    assert torch.isnan(s[rows[:, 0].long()]).tolist() == [False, True, False]
    assert int(q[rows[1, 0]].abs().max()) == 0


# --------------------------------------------------------- weighted sum, back

SUMS = [  # T, k, E, kind, H
    (1, 8, 256, "own", 7168), (61, 6, 20, "any", 1032), (3, 1, 2, "own", 8), (40, 64, 3, "any", 136), (333, 5, 31, "far", 640),
    (17, 9, 30, "own", 4104), (5, 3, 4, "none", 256), (600, 2, 5, "any", 72),
]


def sum_case(T, k, E, kind, H):
    rng = np.random.default_rng(T * 7 + H)
    rows, layout, _ = plan_of(choices(rng, T, k, E, kind), E)
    y = bf16(rng.standard_normal((layout.size, H)))
    y[torch.from_numpy(layout < 0).cuda()] = NAN  # what padding holds is nobody's business
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[rows < 0] = NAN
    return rows, layout, y, w, bf16(rng.standard_normal((T, H)))


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,kind,H", SUMS)
def test_unpermute_matches_definition(T, k, E, kind, H, weighted):
    rows, layout, y, w, _ = sum_case(T, k, E, kind, H)
    got = dg.dg_moe_unpermute(y, to_dev(rows), to_dev(w) if weighted else None)
    want, tol = ref.unpermute(host(y), rows, w if weighted else None)
    assert (np.abs(host(got) - want) <= tol).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,E,kind,H", SUMS)
def test_unpermute_backward_matches_definition(T, k, E, kind, H, weighted):
    rows, layout, y, w, g = sum_case(T, k, E, kind, H)
    wd = to_dev(w) if weighted else None
    some = torch.full((T, k), 5.0, device="cuda")
    want = ref.unpermute_backward(host(g), host(y), rows, w if weighted else None)
    for lay, buf in ((to_dev(layout), None), (None, None), (to_dev(layout), torch.full_like(y, 3.0)),
                     (None, torch.full_like(y, 3.0))):
        gy, gw = dg.dg_moe_unpermute_backward(g, y, to_dev(rows), wd, lay, buf, some)
        pad = layout < 0
        kept = 3.0 if lay is None and buf is not None else 0.0
        assert (host(gy)[pad] == kept).all()
        assert (np.abs(host(gy) - want[0]) <= want[1])[~pad].all()
        assert gw is some and (np.abs(host(gw) - want[2]) <= want[3]).all()
    only_y, none = dg.dg_moe_unpermute_backward(g, y, to_dev(rows), wd, to_dev(layout))
    assert torch.equal(only_y[~torch.from_numpy(pad).cuda()], gy[~torch.from_numpy(pad).cuda()])
    assert (none is None) == (not weighted)


def test_unpermute_takes_rows_outside_the_buffer_as_none():
    y = torch.ones(128, 16, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([[0, 128, -1], [2 ** 31 - 1, -2 ** 31, 127]], dtype=torch.int32, device="cuda")
    assert torch.equal(dg.dg_moe_unpermute(y, rows), torch.ones(2, 16, dtype=torch.bfloat16, device="cuda"))
    gy, gw = dg.dg_moe_unpermute_backward(y[:2].contiguous(), y, rows, torch.full((2, 3), 2.0, device="cuda"))
    assert gw.tolist() == [[16.0, 0.0, 0.0], [0.0, 0.0, 16.0]]
    assert gy.float().sum(1).nonzero().flatten().tolist() == [0, 127] and float(gy.max()) == 2.0


def test_sums_without_sorted_rows_or_without_tokens():
    none = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([[-1, 0], [5, -1]], dtype=torch.int32, device="cuda")
    w = torch.ones(2, 2, device="cuda")
    g = torch.ones(2, 16, dtype=torch.bfloat16, device="cuda")
    assert float(dg.dg_moe_unpermute(none, rows, w).abs().max()) == 0.0
    gy, gw = dg.dg_moe_unpermute_backward(g, none, rows, w)
    assert gy.shape == (0, 16) and float(gw.abs().max()) == 0.0
    y = torch.full((256, 16), 3.0, dtype=torch.bfloat16, device="cuda")
    assert dg.dg_moe_unpermute(y, rows[:0], w[:0]).shape == (0, 16)
    layout = torch.full((256,), -1, dtype=torch.int32, device="cuda")
    layout[7] = 0
    gy, gw = dg.dg_moe_unpermute_backward(g[:0], y, rows[:0], w[:0], layout, y.clone())
    assert gw.shape == (0, 2) and gy.float().sum(1).nonzero().flatten().tolist() == [7]


@pytest.mark.parametrize("value", [INF, NAN])
def test_unpermute_keeps_values_that_are_not_finite_in_their_rows(value):
    rows, layout, y, w, g = sum_case(9, 2, 3, "own", 64)
    y[int(rows[4, 1])] = value
    out = dg.dg_moe_unpermute(y, to_dev(rows), to_dev(w))
    assert (~torch.isfinite(out)).all(1).nonzero().flatten().tolist() == [4]


# ------------------------------------------------------------------ the gate

def gate_case(M, I, seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((M, 2 * I)) * 3
    z[0, :I // 2] = -200 * rng.random(I // 2)
    z[M // 2, :I // 2] = 300 * rng.random(I // 2)
    z[M - 1] = 0
    layout = rng.integers(-1, 3, M).astype(np.int32)
    layout[0] = 0
    return bf16(z), layout, rng


@pytest.mark.parametrize("with_layout", [True, False])
@pytest.mark.parametrize("M,I", [(1, 8), (3, 128), (130, 24), (257, 1416), (64, 2048)])
def test_swiglu_and_gradient_match_definition(M, I, with_layout):
    z, layout, rng = gate_case(M, I, M + I)
    on = layout >= 0 if with_layout else np.ones(M, bool)
    zh = host(z)
    z[torch.from_numpy(~on).cuda()] = NAN
    lay = to_dev(layout) if with_layout else None
    h, err = ref.swiglu(zh)
    d = bf16(rng.standard_normal((M, I)))
    g, gtol = ref.swiglu_backward(zh, host(d))
    for buf in (None, torch.full((M, I), 7.0, dtype=torch.bfloat16, device="cuda")):
        got = dg.dg_swiglu(z, lay, buf)
        assert (np.abs(host(got) - h) <= err + ref.bf16_error(np.abs(h) + err))[on].all() and (host(got)[~on] == 0).all()
        gz = dg.dg_swiglu_backward(z, d, lay, None if buf is None else torch.full_like(z, 7.0))
        assert (np.abs(host(gz) - g) <= gtol)[on].all() and (host(gz)[~on] == 0).all()


@pytest.mark.parametrize("kind", ["fp8", "e8m0", "int8"])
@pytest.mark.parametrize("M,I", [(1, 128), (3, 384), (130, 640), (7, 512), (40, 2048), (9, 2176), (5, 8192), (33, 8320)])
def test_swiglu_quantized_matches_definition(M, I, kind):
    z, layout, _ = gate_case(M, I, M + I)
    zh, on = host(z), layout >= 0
    z[torch.from_numpy(~on).cuda()] = NAN
    h, err = ref.swiglu(zh)
    dt = torch.int8 if kind == "int8" else torch.uint8
    q = torch.full((M, I), 99, dtype=dt, device="cuda")
    shape = {"fp8": (M, I // 128), "e8m0": (M, dg.e8m0_pitch(I // 128)), "int8": (M,)}[kind]
    s = torch.full(shape, 9, dtype=torch.uint8 if kind == "e8m0" else torch.float32, device="cuda")
    call = {"fp8": dg.dg_swiglu_quantize_fp8, "e8m0": dg.dg_swiglu_quantize_fp8_e8m0, "int8": dg.dg_swiglu_quantize_int8}[kind]
    got = call(z, to_dev(layout), q, s)
    assert got[0] is q and got[1] is s
    off = torch.from_numpy(~on).cuda()
    assert bool((q[off] == 99).all()) and bool((s[off] == 9).all())
    qh, sh = q.cpu().numpy()[on], s.cpu().numpy()[on]
    if kind == "int8":
        ref.check_int8(qh.astype(np.float64), sh, h[on], err[on])
    elif kind == "fp8":
        ref.check_fp8(qh, sh, h[on], err[on])
    else:
        kb = I // 128
        assert (sh[:, kb:] == 9).all()
        e = sh[:, :kb].astype(np.float64) - 127
        top = np.abs(h[on]).reshape(-1, kb, 128).max(2)
        slack = 1 + 16 * ref.FP32
        assert (top <= 448 * np.exp2(e) * slack + 1e-36).all()
        assert ((top * slack + 1e-36 > 448 * np.exp2(e - 1)) | (e == -127)).all()
        v = ref.e4m3_value(qh).reshape(-1, kb, 128)
        r = (h[on].reshape(-1, kb, 128)) / np.exp2(e)[:, :, None]
        dr = err[on].reshape(-1, kb, 128) / np.exp2(e)[:, :, None]
        assert (np.abs(v - r) <= ref.e4m3_step(np.minimum(np.abs(r) + dr, 448)) / 2 + dr).all()
    new = call(z, to_dev(layout))
    on_d = torch.from_numpy(on).cuda()
    assert torch.equal(new[0][on_d], q[on_d])
    whole = call(torch.nan_to_num(z))
    assert torch.equal(whole[0][on_d], q[on_d])


@pytest.mark.parametrize("bad", [NAN, INF])
def test_swiglu_marks_blocks_that_are_not_finite(bad):
    z = torch.randn(3, 512, device="cuda").to(torch.bfloat16)
    z[1, 256 + 200] = bad  # in the upper half: the second block's values
    assert torch.isnan(dg.dg_swiglu_quantize_fp8(z)[1]).nonzero().tolist() == [[1, 1]]
    assert (dg.dg_swiglu_quantize_fp8_e8m0(z)[1] == 255).nonzero().tolist() == [[1, 1]]
    q, s = dg.dg_swiglu_quantize_int8(z)
    assert torch.isnan(s).nonzero().tolist() == [[1]] and int(q[1].abs().max()) == 0
