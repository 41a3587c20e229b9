"""CPU tests of include/dg_experts.h and include/dg_int8.h: exported symbols,
refusals (host-side checks that return before anything touches the GPU), the
binding's own checks, and the references' gradients against differences."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from tests import experts_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DG_OK, DG_ERR_NULL, DG_ERR_SHAPE, DG_ERR_ALIGN = 0, 1, 2, 3
FAKE = 0x10000  # 16-byte aligned, never dereferenced: the checks reject first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.library_path()):
        from fp8_block_scaled_gemm_amd import build
        build.build()
    return dg.load_library()


def declared(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(dg_\w+)\s*\(", text)))


@pytest.mark.parametrize("header,count", [("dg_experts.h", 14), ("dg_int8.h", 4)])
def test_every_declared_function_is_exported_and_bound(lib, header, count):
    out = subprocess.run(["nm", "-D", "--defined-only", dg.library_path()], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert len(declared(header)) == count
    for name in declared(header):
        assert name in exported and getattr(lib, name).argtypes, name
        assert name.removesuffix("_bf16") in dg.__all__, name


@pytest.mark.parametrize("header", ["dg_experts.h", "dg_int8.h"])
def test_headers_are_plain_c(header, tmp_path):
    src = tmp_path / "use.c"
    src.write_text(f'#include "{header}"\nint main(void) {{ return (int)DG_OK; }}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", f"-I{ROOT}/include", "-c", str(src), "-o",
                    str(tmp_path / "use.o")], check=True)


BAD_SORTS = [dict(T=-1), dict(k=0), dict(k=65), dict(E=0), dict(E=4097), dict(T=2 ** 30), dict(T=2 ** 62)]


def rows_of(lib, T=4, k=2, E=8):
    n = ctypes.c_int64(-1)
    return lib.dg_moe_sort_rows(T, k, E, ctypes.byref(n)), n.value


def test_sort_sizes(lib):
    for T, k, E in ((0, 1, 1), (1, 8, 256), (4096, 8, 256), (333, 5, 31), (5, 1, 4096)):
        assert rows_of(lib, T, k, E) == (DG_OK, ref.sort_rows(T, k, E)) and dg.dg_moe_sort_rows(T, k, E) == ref.sort_rows(T, k, E)
        assert dg.dg_moe_sort_workspace(T, k, E) >= 0
    for bad in BAD_SORTS:
        assert rows_of(lib, **bad)[0] == DG_ERR_SHAPE, bad
        n = ctypes.c_int64()
        assert lib.dg_moe_sort_workspace(*{**dict(T=4, k=2, E=8), **bad}.values(), ctypes.byref(n)) == DG_ERR_SHAPE
    assert lib.dg_moe_sort_rows(4, 2, 8, None) == DG_ERR_NULL
    assert lib.dg_moe_sort_workspace(4, 2, 8, None) == DG_ERR_NULL
    with pytest.raises(dg.DGError, match="dg_moe_sort_rows"):
        dg.dg_moe_sort_rows(4, 0, 8)


BIG = 100000  # tokens that need the table in the workspace


def test_sort_refusals(lib):
    def call(T=4, k=2, E=8, M=None, ws=FAKE, nbytes=1 << 40, **at):
        p = [at.get(n, FAKE) for n in ("ids", "rows", "layout", "offsets")]
        return lib.dg_moe_sort(*p, T, k, E, (T * k + 127 * E) // 128 * 128 if M is None else M, ws, nbytes, None)
    for bad in BAD_SORTS + [dict(M=1016), dict(M=896), dict(M=1025), dict(M=1 << 31), dict(M=-128)]:
        assert call(**bad) == DG_ERR_SHAPE, bad
    need = dg.dg_moe_sort_workspace(BIG, 2, 8)
    assert need > 0 and call(T=BIG, nbytes=need - 1) == DG_ERR_SHAPE and call(T=BIG, ws=None) == DG_ERR_NULL
    assert call(T=BIG, ws=FAKE + 8) == DG_ERR_ALIGN
    for n in ("ids", "rows", "layout", "offsets"):
        assert call(**{n: None}) == DG_ERR_NULL, n
        assert call(**{n: FAKE + 4}) == DG_ERR_ALIGN, n
    assert call(T=0, offsets=None) == DG_ERR_NULL  # an empty plan is written all the same


@pytest.mark.parametrize("name", ["dg_moe_dispatch", "dg_moe_dispatch_fp8", "dg_moe_dispatch_fp8_e8m0",
                                  "dg_moe_dispatch_int8"])
def test_dispatch_refusals(lib, name):
    names = ["x", "ids", "out"] + ([] if name == "dg_moe_dispatch" else ["s"]) + ["rows", "layout", "offsets"]

    def call(T=4, k=2, E=8, H=256, M=None, ws=FAKE, nbytes=1 << 40, **at):
        M = (T * k + 127 * E) // 128 * 128 if M is None else M
        return getattr(lib, name)(*[at.get(n, FAKE) for n in names], T, k, E, H, M, ws, nbytes, None)
    odd = 12 if name == "dg_moe_dispatch" else 72
    for bad in BAD_SORTS + [dict(M=896), dict(M=1025), dict(H=0), dict(H=odd), dict(H=1 << 24), dict(H=-128)]:
        assert call(**bad) == DG_ERR_SHAPE, bad
    for n in names:
        assert call(**{n: None}) == DG_ERR_NULL, n
        assert call(**{n: FAKE + 4}) == DG_ERR_ALIGN, n
    # copies past the work-items of one grid: refused before the sort is enqueued
    assert call(T=1 << 24, k=64, H=(1 << 24) - 128, E=1) == DG_ERR_SHAPE
    if name == "dg_moe_dispatch":
        assert call(T=4096, k=1, H=(1 << 24) - 128, E=1) == DG_ERR_SHAPE


def test_unpermute_refusals(lib):
    def call(T=4, k=2, H=64, M=128, **at):
        return lib.dg_moe_unpermute(*[at.get(n, FAKE) for n in ("y", "rows", "weights", "out")], T, k, H, M, None)
    bads = [dict(T=-1), dict(T=1 << 31), dict(k=0), dict(k=65), dict(H=0), dict(H=12), dict(H=1 << 24), dict(M=-1),
            dict(M=1 << 31)]
    for bad in bads + [dict(T=(1 << 31) - 1, H=1 << 23)]:
        assert call(**bad) == DG_ERR_SHAPE, bad
    for n in ("y", "rows", "out"):
        assert call(**{n: None}) == DG_ERR_NULL, n
    for n in ("y", "rows", "out", "weights"):
        assert call(**{n: FAKE + 4}) == DG_ERR_ALIGN, n
    assert call(T=0, y=None, rows=None, out=None) == DG_OK

    names = ("grad", "y", "rows", "weights", "layout", "grad_y", "grad_weights")

    def back(T=4, k=2, H=64, M=128, **at):
        return lib.dg_moe_unpermute_backward(*[at.get(n, FAKE) for n in names], T, k, H, M, None)
    for bad in bads + [dict(T=(1 << 31) - 1)]:
        assert back(**bad) == DG_ERR_SHAPE, bad
    for n in ("grad", "rows", "y"):
        assert back(**{n: None}) == DG_ERR_NULL, n
    assert back(grad_y=None, grad_weights=None) == DG_ERR_NULL
    for n in names:
        assert back(**{n: FAKE + 4}) == DG_ERR_ALIGN, n
    assert back(T=0, M=0, grad=None, rows=None, grad_y=None, grad_weights=None) == DG_OK


@pytest.mark.parametrize("name", ["dg_swiglu", "dg_swiglu_quantize_fp8", "dg_swiglu_quantize_fp8_e8m0",
                                  "dg_swiglu_quantize_int8", "dg_swiglu_backward"])
def test_swiglu_refusals(lib, name):
    names = {"dg_swiglu": ["z", "layout", "h"], "dg_swiglu_backward": ["z", "grad", "layout", "out"]}.get(
        name, ["z", "layout", "q", "s"])

    def call(M=4, I=256, **at):
        return getattr(lib, name)(*[at.get(n, FAKE) for n in names], M, I, None)
    odd = 72 if "quantize" in name else 12
    for bad in (dict(M=-1), dict(M=1 << 31), dict(I=0), dict(I=odd), dict(I=1 << 23), dict(M=(1 << 31) - 1, I=(1 << 23) - 128)):
        assert call(**bad) == DG_ERR_SHAPE, bad
    for n in names:
        if n != "layout":
            assert call(**{n: None}) == DG_ERR_NULL, n
        assert call(**{n: FAKE + 4}) == DG_ERR_ALIGN, n
    assert call(M=0, **{n: None for n in names}) == DG_OK


def test_int8_refusals(lib):
    names = ("A", "sa", "B", "sb", "D")

    def dense(M=4, N=16, K=128, **at):
        return lib.dg_int8_gemm_nt(*[at.get(n, FAKE) for n in names], M, N, K, None)

    def grouped(M=128, N=16, K=128, G=2, **at):
        return lib.dg_int8_gemm_grouped_contiguous(*[at.get(n, FAKE) for n in names + ("layout",)], M, N, K, G, None)
    for call in (dense, grouped):
        for bad in (dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=12), dict(N=1 << 31), dict(K=0), dict(K=100),
                    dict(K=1 << 17)):
            assert call(**bad) == DG_ERR_SHAPE, bad
        for n in names:
            assert call(**{n: None}) == DG_ERR_NULL, n
            assert call(**{n: FAKE + 4}) == DG_ERR_ALIGN, n
        assert call(M=0, **{n: None for n in names}) == DG_OK
    assert dense(M=(1 << 31) - 128, N=1 << 30) == DG_ERR_SHAPE  # more tiles than a grid holds
    for bad in (dict(M=130), dict(G=0), dict(G=1 << 31)):
        assert grouped(**bad) == DG_ERR_SHAPE, bad
    assert grouped(layout=None) == DG_ERR_NULL and grouped(layout=FAKE + 8) == DG_ERR_ALIGN
    for name in ("dg_quantize_int8_per_row", "dg_quantize_int8_per_row_bf16"):
        f = getattr(lib, name)
        for M, K in ((-1, 128), (4, 0), (4, 64), (4, 1 << 24), (1 << 26, 128), (1 << 24, 4096), (1 << 62, 128)):
            assert f(FAKE, M, K, FAKE, FAKE, None) == DG_ERR_SHAPE, (M, K)
        assert f(None, 4, 128, FAKE, FAKE, None) == DG_ERR_NULL and f(FAKE, 4, 128, FAKE, FAKE + 4, None) == DG_ERR_ALIGN
        assert f(None, 0, 128, None, None, None) == DG_OK


def test_binding_refuses_host_tensors_and_wrong_kinds(lib):
    x, ids = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    q = torch.zeros(4, 128, dtype=torch.int8)
    for call in (lambda: dg.dg_moe_sort(ids, 4), lambda: dg.dg_moe_dispatch(x, ids, 4), lambda: dg.dg_moe_dispatch_fp8(x, ids, 4),
                 lambda: dg.dg_moe_dispatch_fp8_e8m0(x, ids, 4), lambda: dg.dg_moe_dispatch_int8(x, ids, 4),
                 lambda: dg.dg_moe_unpermute(x, ids), lambda: dg.dg_moe_unpermute_backward(x, x, ids), lambda: dg.dg_swiglu(x),
                 lambda: dg.dg_swiglu_quantize_fp8(x), lambda: dg.dg_swiglu_quantize_fp8_e8m0(x),
                 lambda: dg.dg_swiglu_quantize_int8(x), lambda: dg.dg_swiglu_backward(x, x),
                 lambda: dg.dg_int8_gemm_nt(q, None, q, None, None),
                 lambda: dg.dg_int8_gemm_grouped_contiguous(q, None, q, None, None, ids), lambda: dg.dg_quantize_int8_per_row(x)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
    with pytest.raises(ValueError, match="dimensions"):
        dg.dg_moe_sort(ids[0], 4)
    with pytest.raises(TypeError):
        dg.dg_moe_sort([[1]], 4)
    with pytest.raises(TypeError, match="grouped_layout"):
        dg.dg_int8_gemm_grouped_contiguous(q, None, q, None, None, None)


def test_reference_gradients_match_differences():
    """The formulas that the kernels are held to, against central differences
    of the definitions, in 64 bits."""
    rng = np.random.default_rng(2)
    step = 1e-6

    def differences(f, at):
        out = np.zeros_like(at)
        for i in np.ndindex(*at.shape):
            up, down = at.copy(), at.copy()
            up[i] += step
            down[i] -= step
            out[i] = (f(up) - f(down)) / (2 * step)
        return out
    y, w, g = rng.standard_normal((9, 4)), rng.standard_normal((5, 2)), rng.standard_normal((5, 4))
    rows = np.array([[0, 3], [-1, 5], [8, 1], [2, 9], [7, -1]], np.int32)
    gy, _, gw, _ = ref.unpermute_backward(g, y, rows, w)
    assert np.abs(gy - differences(lambda v: (ref.unpermute(v, rows, w)[0] * g).sum(), y)).max() < 1e-8
    # the weights enter the reference as they are held, in 64 bits here
    assert np.abs(gw - differences(lambda v: (ref.unpermute(y, rows, v)[0] * g).sum(), w)).max() < 1e-8
    z, d = rng.standard_normal((3, 12)) * 2, rng.standard_normal((3, 6))
    want = differences(lambda v: (ref.swiglu(v)[0] * d).sum(), z)
    assert np.abs(ref.swiglu_backward(z, d)[0] - want).max() < 1e-8
