"""CPU tests of include/dg_ops.h: exported symbols, refusals (host-side checks
that return before anything touches the GPU) and the binding's own checks."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import fp8_block_scaled_gemm_amd as dg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DG_OK, DG_ERR_NULL, DG_ERR_SHAPE, DG_ERR_ALIGN, DG_ERR_UNSUPPORTED = 0, 1, 2, 3, 4
FAKE = 0x10000  # 16-byte aligned, never dereferenced: the checks reject first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.library_path()):
        from fp8_block_scaled_gemm_amd import build
        build.build()
    return dg.load_library()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "dg_ops.h")).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(dg_\w+)\s*\(", text)))


def test_every_declared_function_is_exported_and_bound(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", dg.library_path()], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert len(declared()) == 10
    for name in declared():
        assert name in exported, name
        assert getattr(lib, name).argtypes, name


def _topk(lib, name="dg_moe_topk", x=FAKE, bias=None, ids=FAKE, w=FAKE, T=4, E=16, k=2, g=1, tg=1, mode=0):
    return getattr(lib, name)(x, bias, ids, w, T, E, k, g, tg, mode, 1, 1.0, None)


@pytest.mark.parametrize("name", ["dg_moe_topk", "dg_moe_topk_bf16"])
def test_topk_refusals(lib, name):
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=65, E=128), dict(k=17),
                dict(g=0), dict(g=3), dict(g=128, E=128), dict(g=4, tg=0), dict(g=4, tg=5),
                dict(g=4, tg=1, k=5), dict(T=1 << 61)):
        assert _topk(lib, name, **bad) == DG_ERR_SHAPE, bad
    assert _topk(lib, name, mode=2) == DG_ERR_UNSUPPORTED
    assert _topk(lib, name, x=None) == DG_ERR_NULL
    assert _topk(lib, name, w=None) == DG_ERR_NULL
    assert _topk(lib, name, ids=FAKE + 4) == DG_ERR_ALIGN
    assert _topk(lib, name, bias=FAKE + 4) == DG_ERR_ALIGN
    assert _topk(lib, name, x=None, ids=None, w=None, T=0) == DG_OK
    assert _topk(lib, name, T=1 << 40) == DG_ERR_SHAPE  # more than 2^31 - 1 workgroups


@pytest.mark.parametrize("name", ["dg_moe_topk_backward", "dg_moe_topk_backward_bf16"])
def test_topk_backward_refusals(lib, name):
    def call(x=FAKE, ids=FAKE, g=FAKE, out=FAKE, T=4, E=16, k=2, mode=1):
        return getattr(lib, name)(x, ids, g, out, T, E, k, mode, 1, 1.0, None)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=65)):
        assert call(**bad) == DG_ERR_SHAPE, bad
    assert call(mode=-1) == DG_ERR_UNSUPPORTED
    assert call(out=None) == DG_ERR_NULL
    assert call(g=FAKE + 8) == DG_ERR_ALIGN
    assert call(x=None, ids=None, g=None, out=None, T=0) == DG_OK


def _moe_bytes(lib, T=4, k=2, E=8, H=256, I=128):
    n = ctypes.c_int64(-1)
    return lib.dg_moe_mlp_fp8_workspace(T, k, E, H, I, ctypes.byref(n)), n.value


@pytest.mark.parametrize("name", ["dg_moe_mlp_fp8", "dg_moe_mlp_fp8_e8m0"])
def test_moe_refusals(lib, name):
    def call(T=4, k=2, E=8, H=256, I=128, ws=FAKE, nbytes=None, **at):
        p = [at.get(n, FAKE) for n in ("x", "sx", "ids", "weights", "w13", "s13", "w2", "s2", "y")]
        if nbytes is None:
            nbytes = 1 << 40
        return getattr(lib, name)(*p, T, k, E, H, I, ws, nbytes, None)
    for bad in (dict(T=-1), dict(T=257), dict(k=0), dict(k=17), dict(E=0), dict(E=65537), dict(H=0),
                dict(H=200), dict(H=16512), dict(I=-128), dict(I=64), dict(I=16512)):
        assert call(**bad) == DG_ERR_SHAPE, bad
        n = ctypes.c_int64()
        sizes = {**dict(T=4, k=2, E=8, H=256, I=128), **bad}
        assert lib.dg_moe_mlp_fp8_workspace(*sizes.values(), ctypes.byref(n)) == DG_ERR_SHAPE
    status, need = _moe_bytes(lib)
    assert status == DG_OK and need > 0
    assert call(nbytes=need - 1) == DG_ERR_SHAPE
    for n in ("x", "sx", "ids", "weights", "w13", "s13", "w2", "s2", "y"):
        assert call(**{n: None}) == DG_ERR_NULL, n
        assert call(**{n: FAKE + 4}) == DG_ERR_ALIGN, n
    assert call(ws=None) == DG_ERR_NULL
    assert call(ws=FAKE + 8) == DG_ERR_ALIGN
    assert call(T=0, x=None, y=None, ws=None, nbytes=0) == DG_OK
    assert lib.dg_moe_mlp_fp8_workspace(4, 2, 8, 256, 128, None) == DG_ERR_NULL


def test_moe_workspace_grows_with_the_pairs(lib):
    sizes = [_moe_bytes(lib, T=T, k=k)[1] for T, k in ((1, 1), (4, 2), (64, 8), (256, 16))]
    assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.parametrize("name", ["dg_fp8_gemm_nt_lora", "dg_fp8_gemm_nt_lora_e8m0"])
def test_lora_refusals(lib, name):
    names = ("A", "sa", "B", "sb", "D", "x", "la", "lb", "ids", "scaling")

    def call(M=4, N=16, K=128, L=2, R=8, ws=FAKE, nbytes=1 << 40, **at):
        return getattr(lib, name)(*[at.get(n, FAKE) for n in names], M, N, K, L, R, ws, nbytes, None)
    for bad in (dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=12), dict(N=1 << 22), dict(K=0), dict(K=100),
                dict(K=1 << 24), dict(L=0), dict(L=65537), dict(R=0), dict(R=12), dict(R=136)):
        assert call(**bad) == DG_ERR_SHAPE, bad
    n = ctypes.c_int64()
    assert lib.dg_fp8_gemm_nt_lora_workspace(4, 16, 128, 2, 8, ctypes.byref(n)) == DG_OK and n.value >= 4 * 8 * 4
    assert call(nbytes=n.value - 1) == DG_ERR_SHAPE
    for p in names:
        assert call(**{p: None}) == DG_ERR_NULL, p
        assert call(**{p: FAKE + 4}) == DG_ERR_ALIGN, p
    assert call(ws=None) == DG_ERR_NULL
    assert call(M=0, A=None, D=None, ws=None, nbytes=0) == DG_OK
    assert lib.dg_fp8_gemm_nt_lora_workspace(4, 16, 128, 2, 12, ctypes.byref(n)) == DG_ERR_SHAPE
    assert lib.dg_fp8_gemm_nt_lora_workspace(4, 16, 128, 2, 8, None) == DG_ERR_NULL


def test_binding_refuses_host_tensors_and_bad_modes(lib):
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="on the GPU"):
        dg.dg_moe_topk(x, 2)
    with pytest.raises(ValueError, match="dimensions"):
        dg.dg_moe_topk(torch.zeros(16), 2)
    with pytest.raises(TypeError):
        dg.dg_moe_topk([[1.0]], 1)
    with pytest.raises(ValueError, match="on the GPU"):
        dg.dg_moe_topk_backward(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    c = torch.zeros(4, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="on the GPU"):
        dg.dg_moe_mlp_fp8(c, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="on the GPU"):
        dg.dg_fp8_gemm_nt_lora(c, None, c, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="scoring"):
        dg._score_mode("relu")


@pytest.mark.parametrize("name", ["dg_fp8_gemm_nt_lora", "dg_fp8_gemm_nt_lora_e8m0"])
def test_lora_refuses_a_grid_too_large_before_the_first_launch(lib, name):
    M, N = 2 ** 31 - 1, 2 ** 22 - 8
    n = ctypes.c_int64(-1)
    assert lib.dg_fp8_gemm_nt_lora_workspace(M, N, 128, 2, 8, ctypes.byref(n)) == DG_ERR_SHAPE and n.value == -1
    assert getattr(lib, name)(*[FAKE] * 10, M, N, 128, 2, 8, FAKE, 1 << 60, None) == DG_ERR_SHAPE
