"""The operators of include/dg_ops.h on the GPU against their 64-bit
definitions (tests/ops_ref.py), at the sizes and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import ops_ref as ref
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def to_bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


# ----------------------------------------------------------------- router

def logits_of(rng, T, E, dtype, pattern):
    x = rng.standard_normal((T, E)).astype(np.float32) * 3
    if pattern == "masked":
        x[rng.random((T, E)) < 0.6] = -INF
        x[0] = -INF                        # no expert open at all
        x[T // 2, :] = NAN
        x[T - 1, E // 2] = INF
    elif pattern == "ties":
        x = np.round(x)
        x[0] = 0.0
        x[T - 1] = np.where(np.arange(E) % 2, -0.0, 0.0)
    elif pattern == "extreme":
        x[0] = np.finfo(np.float32).min
        x[T // 2] = -100.0
        x[T - 1, :2] = INF
        x[T - 1, 2:] = np.finfo(np.float32).min
    t = torch.from_numpy(x)
    return t.to(torch.bfloat16) if dtype == "bf16" else t


ROUTERS = [  # T, E, k, n_group, topk_group, scoring, renorm, bias, dtype, pattern
    (1, 256, 8, 8, 4, "sigmoid", True, True, "fp32", "plain"),
    (5, 256, 8, 8, 4, "sigmoid", True, True, "fp32", "masked"),
    (37, 256, 8, 8, 3, "softmax", True, True, "bf16", "plain"),
    (3, 1, 1, 1, 1, "softmax", True, False, "fp32", "plain"),
    (9, 61, 5, 1, 1, "softmax", False, False, "fp32", "masked"),
    (9, 61, 61, 1, 1, "sigmoid", True, False, "bf16", "masked"),
    (130, 128, 8, 1, 1, "softmax", True, False, "bf16", "ties"),
    (7, 96, 6, 4, 2, "softmax", False, False, "fp32", "ties"),
    (7, 60, 4, 3, 2, "sigmoid", False, True, "fp32", "masked"),
    (6, 512, 16, 16, 2, "sigmoid", True, False, "fp32", "plain"),
    (6, 1000, 64, 1, 1, "sigmoid", True, True, "fp32", "masked"),
    (6, 1024, 7, 64, 64, "softmax", True, True, "fp32", "plain"),
    (8, 64, 8, 1, 1, "softmax", True, False, "fp32", "extreme"),
    (8, 64, 8, 8, 8, "sigmoid", True, True, "fp32", "extreme"),
    (8, 16, 2, 16, 4, "sigmoid", True, True, "fp32", "plain"),
]


@pytest.mark.parametrize("T,E,k,G,tg,scoring,renorm,bias,dtype,pattern", ROUTERS)
def test_topk_matches_definition(T, E, k, G, tg, scoring, renorm, bias, dtype, pattern):
    rng = np.random.default_rng(T * 1000 + E)
    x = logits_of(rng, T, E, dtype, pattern)
    b = rng.standard_normal(E).astype(np.float32) * 0.2 if bias else None
    if bias and pattern == "masked":
        b[E - 1], b[0] = -INF, NAN
    ids, w = dg.dg_moe_topk(x.cuda(), k, bias=None if b is None else to_dev(b), n_group=G, topk_group=tg,
                            scoring=scoring, renormalize=renorm, scale=1.5)
    want_ids, want_w = ref.topk(x.float().numpy(), b, k, G, tg, scoring, renorm, 1.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # exp of a difference rounded to fp32, its own rounding, sums and divisions
    finite = x.float().numpy()[np.isfinite(x.float().numpy()) & (np.abs(x.float().numpy()) < 1e30)]
    spread = 2 * float(np.abs(finite).max()) if finite.size else 0.0
    tol = (spread + 32) * 2 * ref.FP32 * np.abs(want_w) + 1e-37
    assert (np.abs(host(w) - want_w) <= tol).all()


def test_topk_no_rows_and_given_outputs():
    ids, w = dg.dg_moe_topk(torch.zeros(0, 16, device="cuda"), 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)
    x = torch.randn(6, 40, device="cuda")
    ids = torch.full((6, 4), 77, dtype=torch.int32, device="cuda")
    w = torch.full((6, 4), NAN, device="cuda")
    got = dg.dg_moe_topk(x, 4, ids, w)
    assert got[0] is ids and got[1] is w
    assert int(ids.max()) < 40 and bool(torch.isfinite(w).all())


@pytest.mark.parametrize("T,E,k,scoring,renorm,dtype,pattern", [
    (1, 256, 8, "sigmoid", True, "fp32", "plain"), (33, 61, 5, "sigmoid", True, "fp32", "masked"),
    (33, 61, 5, "softmax", True, "bf16", "masked"), (130, 128, 8, "softmax", False, "fp32", "plain"),
    (5, 1000, 64, "softmax", True, "fp32", "plain"), (7, 300, 1, "softmax", False, "bf16", "plain"),
    (8, 64, 8, "softmax", True, "fp32", "extreme"), (8, 64, 8, "sigmoid", False, "fp32", "extreme")])
def test_topk_backward_matches_formula(T, E, k, scoring, renorm, dtype, pattern):
    rng = np.random.default_rng(T + E)
    x = logits_of(rng, T, E, dtype, pattern)
    ids, _ = ref.topk(x.float().numpy(), None, k, 1, 1, scoring, renorm, 1.0)
    if pattern == "masked":  # entries of another GPU's experts, and an expert listed twice
        ids[1, 0], ids[2, 1] = E + 5, -7
        ids[3, 1] = ids[3, 0]
    gw = rng.standard_normal((T, k)).astype(np.float32)
    got = dg.dg_moe_topk_backward(x.cuda(), to_dev(ids), to_dev(gw), scoring=scoring, renormalize=renorm,
                                  scale=2.5)
    want, mag = ref.topk_backward(x.float().numpy(), ids, gw, scoring, renorm, 2.5)
    tol = 128 * ref.FP32 * mag + 1e-37 + (ref.BF16 * np.abs(want) if dtype == "bf16" else 0)
    assert got.dtype == x.dtype
    assert (np.abs(host(got) - want) <= tol).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_topk_backward_matches_differences(scoring, renorm):
    """Central differences, in 64 bits, of the weights the definition gives."""
    rng = np.random.default_rng(5)
    T, E, k, step = 3, 20, 4, 1e-5
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids, _ = ref.topk(x, None, k, 1, 1, scoring, renorm, 1.0)
    gw = rng.standard_normal((T, k)).astype(np.float32)
    want = np.zeros((T, E))
    for e in range(E):
        up, down = x.astype(np.float64), x.astype(np.float64)
        up[:, e] += step
        down[:, e] -= step
        d = ref.topk_weights(up, ids, scoring, renorm, 1.3) - ref.topk_weights(down, ids, scoring, renorm, 1.3)
        want[:, e] = (d * gw).sum(1) / (2 * step)
    got = dg.dg_moe_topk_backward(to_dev(x), to_dev(ids), to_dev(gw), scoring=scoring, renormalize=renorm, scale=1.3)
    # the differences' own error is of order step^2 and 1e-16 / step
    assert np.abs(host(got) - want).max() <= 1e-8 + 128 * ref.FP32 * np.abs(gw).sum(1).max() * 2


# ------------------------------------------------------------ expert layer

def moe_case(seed, T, k, E, H, I, kind, local=None):
    rng = np.random.default_rng(seed)
    spread = local or E
    x = to_bf16(rng.standard_normal((T, H))).float().numpy()
    xq, sx = ref.quantize_rows(x, kind)
    w13 = [ref.quantize_blocks(rng.standard_normal((2 * I, H)) * H ** -0.5, kind) for _ in range(E)]
    w2 = [ref.quantize_blocks(rng.standard_normal((H, I)) * I ** -0.5, kind) for _ in range(E)]
    ids = np.stack([rng.permutation(max(spread, k))[:k] for _ in range(T)]).astype(np.int32)
    ids[ids >= E] = -1
    w = rng.random((T, k)).astype(np.float32) + 0.1
    return dict(x=xq, sx=sx, ids=ids, weights=w, w13=np.stack([q for q, _ in w13]),
                s13=np.stack([s for _, s in w13]), w2=np.stack([q for q, _ in w2]),
                s2=np.stack([s for _, s in w2]))


MOE_ORDER = ("x", "sx", "ids", "weights", "w13", "s13", "w2", "s2")


def run_moe(c, kind, **more):
    call = dg.dg_moe_mlp_fp8 if kind == "fp32" else dg.dg_moe_mlp_fp8_e8m0
    return call(*[to_dev(c[n]) for n in MOE_ORDER], **more)


def check_moe(c, kind):
    got = host(run_moe(c, kind))
    want, tol = ref.moe(*[c[n] for n in MOE_ORDER], kind)
    tol = tol + ref.BF16 * (np.abs(want) + tol) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} out, worst {np.abs(got - want).max()}"


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("T,k,E,H,I,local", [
    (1, 1, 1, 128, 128, None), (1, 8, 16, 256, 256, None), (1, 2, 3, 640, 384, None),
    (3, 2, 5, 640, 384, None), (16, 2, 4, 256, 128, None), (17, 3, 4, 384, 256, None),
    (33, 2, 2, 256, 128, None), (64, 4, 6, 256, 256, None), (65, 1, 2, 128, 128, None),
    (100, 1, 1, 256, 128, None), (40, 8, 300, 128, 128, None), (64, 6, 8, 256, 128, 64),
    (256, 8, 3, 128, 128, 24), (256, 16, 20, 128, 128, None)])
def test_moe_matches_definition(T, k, E, H, I, local, kind):
    check_moe(moe_case(T * 31 + E, T, k, E, H, I, kind, local), kind)


@pytest.mark.parametrize("T", [2, 20, 70])
def test_moe_ids_elsewhere_repeated_and_all_on_one(T):
    c = moe_case(7, T, 3, 5, 256, 256, "fp32")
    c["ids"][0] = [-1, 5, 1 << 30]         # no expert here
    c["ids"][1] = [2, 2, 2]                # one expert three times
    check_moe(c, "fp32")
    assert (host(run_moe(c, "fp32"))[0] == 0).all()
    c["ids"][:] = 4                        # every pair on one expert: T * 3 rows
    check_moe(c, "fp32")
    c["ids"][:] = -1
    assert (host(run_moe(c, "fp32")) == 0).all()


def test_moe_bits_are_reproducible_and_outputs_whole():
    c = moe_case(8, 48, 4, 7, 384, 256, "fp32")
    y = torch.full((48, 384), NAN, dtype=torch.bfloat16, device="cuda")
    first = run_moe(c, "fp32", y=y)
    assert first is y and bool(torch.isfinite(y).all())
    ws = torch.full((dg._workspace_bytes("dg_moe_mlp_fp8_workspace", 48, 4, 7, 384, 256),), 255,
                    dtype=torch.uint8, device="cuda")
    assert torch.equal(run_moe(c, "fp32", workspace=ws), y)
    with pytest.raises(dg.DGError):
        run_moe(c, "fp32", workspace=ws[:-16])


def test_moe_no_tokens():
    c = moe_case(9, 1, 2, 3, 128, 128, "fp32")
    d = {n: to_dev(v) for n, v in c.items()}
    y = dg.dg_moe_mlp_fp8(d["x"][:0], d["sx"][:0], d["ids"][:0], d["weights"][:0], d["w13"], d["s13"], d["w2"], d["s2"])
    assert y.shape == (0, 128)


# --------------------------------------------------------- low-rank adapters

def lora_case(seed, M, N, K, R, L, kind, rows="mixed"):
    rng = np.random.default_rng(seed)
    xb = to_bf16(rng.standard_normal((M, K)))
    x = xb.float().numpy()
    A, sa = ref.quantize_rows(x, kind)
    B, sb = ref.quantize_blocks(rng.standard_normal((N, K)) * K ** -0.5, kind)
    if rows == "each":
        ids = np.arange(M) % (L + 1) - 1
    elif rows == "runs":
        ids = (np.arange(M) // 37) % (L + 2) - 1   # also an id past the last adapter
    elif rows == "none":
        ids = np.full(M, -1)
    else:
        ids = rng.integers(-1, L, M)
    return dict(A=A, sa=sa, B=B, sb=sb, x=xb, la=to_bf16(rng.standard_normal((L, R, K)) * K ** -0.5),
                lb=to_bf16(rng.standard_normal((L, N, R)) * R ** -0.5), ids=ids.astype(np.int32),
                scaling=(rng.random(L) + 0.5).astype(np.float32))


def run_lora(c, kind, **more):
    call = dg.dg_fp8_gemm_nt_lora if kind == "fp32" else dg.dg_fp8_gemm_nt_lora_e8m0
    D = torch.full((c["A"].shape[0], c["B"].shape[0]), NAN, dtype=torch.bfloat16, device="cuda")
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else to_dev(v) for n, v in c.items()}
    got = call(d["A"], d["sa"], d["B"], d["sb"], D, d["x"], d["la"], d["lb"], d["ids"], d["scaling"], **more)
    assert got is D
    return D


def lora_ref(c, kind):
    f = lambda t: t.double().numpy()  # noqa: E731
    return ref.lora(c["A"], c["sa"], c["B"], c["sb"], f(c["x"]), f(c["la"]), f(c["lb"]), c["ids"],
                    c["scaling"].astype(np.float64), kind)


def check_lora(c, kind, rows=None):
    got = host(run_lora(c, kind))
    want, tol = lora_ref(c, kind)
    if rows is not None:
        got, want, tol = got[rows], want[rows], tol[rows]
    tol = tol + ref.BF16 * (np.abs(want) + tol) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} out, worst {np.abs(got - want)[bad].max()}"


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("M,N,K,R,L,rows", [
    (1, 8, 128, 8, 1, "mixed"), (1, 520, 256, 16, 4, "each"), (2, 136, 640, 24, 3, "each"),
    (16, 264, 384, 64, 20, "each"), (17, 1024, 128, 128, 2, "mixed"), (33, 72, 1152, 32, 5, "mixed"),
    (64, 256, 512, 40, 64, "each"), (65, 128, 256, 16, 3, "runs"), (130, 392, 256, 72, 7, "mixed"),
    (300, 520, 384, 24, 4, "runs"), (257, 264, 128, 8, 300, "each"), (20, 64, 128, 16, 2, "none")])
def test_lora_matches_definition(M, N, K, R, L, rows, kind):
    check_lora(lora_case(M * 7 + N, M, N, K, R, L, kind, rows), kind)


@pytest.mark.parametrize("shape", ["256x256", "256x224", "256x192", "256x160", "128x256", "128x128",
                                   "128x64", "128x32", "256x256t"])
def test_lora_every_tile_shape(shape, monkeypatch):
    monkeypatch.setenv("DG_FP8_DENSE_TILE", shape)
    kind = "e8m0" if shape.endswith("t") else "fp32"
    check_lora(lora_case(3, 300, 328, 256, 40, 5, kind, "mixed"), kind)


@pytest.mark.parametrize("M", [6, 200])
def test_lora_one_requests_infinities_stay_its_own(M):
    c = lora_case(11, M, 136, 256, 16, 4, "fp32", "each")
    c["la"][1, 3, 7] = INF
    c["lb"][2] = NAN
    c["scaling"][3] = INF
    c["x"][5, 9] = NAN                     # row 5 has no adapter: x is not read for it
    c["ids"][5] = -1
    clean = np.isin(c["ids"], [-1, 0])
    assert clean.any() and not clean.all()
    check_lora(c, "fp32", rows=clean)
    got = host(run_lora(c, "fp32"))
    assert np.isnan(got[c["ids"] == 2]).all()
    assert not np.isfinite(got[c["ids"] == 3]).any()


def test_lora_without_adapters_is_the_dense_product():
    for M in (9, 140):
        c = lora_case(12, M, 264, 384, 16, 3, "fp32", "none")
        D = torch.empty(M, 264, dtype=torch.bfloat16, device="cuda")
        dg.dg_fp8_gemm_nt(*[to_dev(c[n]) for n in ("A", "sa", "B", "sb")], D)
        want, tol = lora_ref(c, "fp32")
        assert (np.abs(host(run_lora(c, "fp32")) - host(D)) <= 2 * (tol + ref.BF16 * np.abs(want))).all()


# ------------------------------------------------ streams, graphs, refusals

def every_operator():
    """Small calls of every operator on fixed inputs: name -> function of no arguments."""
    rng = np.random.default_rng(21)
    x = torch.from_numpy(rng.standard_normal((40, 64)).astype(np.float32)).cuda()
    ids, _ = dg.dg_moe_topk(x, 4)
    gw = torch.from_numpy(rng.standard_normal((40, 4)).astype(np.float32)).cuda()
    m = {n: to_dev(v) for n, v in moe_case(22, 20, 3, 4, 256, 256, "fp32").items()}
    lo = {}
    for M in (20, 200):
        c = lora_case(23, M, 264, 256, 24, 3, "fp32")
        d = {n: v.cuda() if isinstance(v, torch.Tensor) else to_dev(v) for n, v in c.items()}
        d["D"] = torch.empty(M, 264, dtype=torch.bfloat16, device="cuda")
        lo[M] = d
    args = ("A", "sa", "B", "sb", "D", "x", "la", "lb", "ids", "scaling")
    return {
        "topk": lambda: dg.dg_moe_topk(x, 4, scoring="sigmoid", n_group=4, topk_group=2),
        "topk_backward": lambda: dg.dg_moe_topk_backward(x, ids, gw),
        "moe": lambda: dg.dg_moe_mlp_fp8(*[m[n] for n in MOE_ORDER]),
        "lora_few": lambda: dg.dg_fp8_gemm_nt_lora(*[lo[20][n] for n in args]),
        "lora_many": lambda: dg.dg_fp8_gemm_nt_lora(*[lo[200][n] for n in args]),
    }


def _copies(v):
    return [t.clone() for t in (v if isinstance(v, tuple) else (v,))]


@pytest.mark.parametrize("name", ["topk", "topk_backward", "moe", "lora_few", "lora_many"])
def test_graph_replays_match_eager(name):
    call = every_operator()[name]
    eager = _copies(call())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    out = out if isinstance(out, tuple) else (out,)
    for _ in range(3):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, e in zip(out, eager):
            assert torch.equal(o, e)
        call()  # eager work between replays
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["topk", "topk_backward", "moe", "lora_few", "lora_many"])
def test_runs_on_the_current_stream(name):
    call = every_operator()[name]
    want = _copies(call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _copies(call())
    torch.cuda.current_stream().wait_stream(side)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_binding_refusals():
    x = torch.randn(4, 16, device="cuda")
    with pytest.raises(TypeError):
        dg.dg_moe_topk(x.double(), 2)
    with pytest.raises(ValueError, match="contiguous"):
        dg.dg_moe_topk(torch.randn(16, 4, device="cuda").t(), 2)
    with pytest.raises(ValueError, match="shape"):
        dg.dg_moe_topk(x, 2, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(dg.DGError):
        dg.dg_moe_topk(x, 17)
    with pytest.raises(ValueError, match="scoring"):
        dg.dg_moe_topk(x, 2, scoring="tanh")
    c = lora_case(1, 4, 16, 128, 8, 2, "fp32")
    c["ids"] = c["ids"][:3]
    with pytest.raises(ValueError, match="shape"):
        run_lora(c, "fp32")
    m = moe_case(1, 2, 2, 3, 128, 128, "fp32")
    m["sx"] = m["sx"].astype(np.float64)
    with pytest.raises(TypeError):
        run_moe(m, "fp32")


@pytest.mark.parametrize("kind", ["fp32", "e8m0"])
@pytest.mark.parametrize("T", [2, 12, 40])
def test_moe_infinities_and_nans_stay_in_their_tokens(T, kind):
    """A NaN code, or an activation that overflows, makes its token's row NaN and no other."""
    c = moe_case(13, T, 2, 3, 256, 512, kind)
    want, tol = ref.moe(*[c[n] for n in MOE_ORDER], kind)
    c["x"][1, 77] = 0x7F                   # NaN
    if T > 2:
        c["sx"][5, :] = 254 if kind == "e8m0" else 3e38   # gate * up is past the largest fp32
    got = host(run_moe(c, kind))
    hit = np.zeros(T, bool)
    hit[1] = True
    hit[5:6] = T > 2
    assert np.isnan(got[hit]).all()
    assert (np.abs(got - want)[~hit] <= (tol + ref.BF16 * (np.abs(want) + tol))[~hit]).all()


def test_moe_zero_rows_give_zeros():
    for T in (3, 30):
        c = moe_case(14, T, 2, 3, 128, 256, "fp32")
        c["x"][0] = 0
        c["sx"][0] = 0
        assert (host(run_moe(c, "fp32"))[0] == 0).all()
        check_moe(c, "fp32")
