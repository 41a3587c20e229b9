"""MI355X (gfx950) FP8 block-scaled NT GEMM: thin Python binding.

Every function here has the name of the C-ABI entry point it calls
(include/dg_fp8.h, dg_ops.h, dg_experts.h, dg_int8.h) and only marshals
arguments: it checks torch tensor dtypes, shapes and devices, passes raw device
pointers and the current HIP stream, and raises ``DGError`` on a nonzero status.
For the operators of the last three a compiled extension, ``_binding.so``, does so.  All
arithmetic runs in the HIP kernels of ``libdgfp8.so``; there is no CPU
fallback, and a call fails loudly when the library has not been built
(``python -m fp8_block_scaled_gemm_amd.build``).

Tensor conventions: e4m3 codes are ``torch.uint8`` (or
``torch.float8_e4m3fn``, viewed as bytes), scales ``torch.float32``, int8 codes
``torch.int8``, group arrays ``torch.int32``, and D is ``torch.bfloat16`` (or ``torch.uint16`` /
``torch.int16`` holding bf16 bit patterns).  All tensors live on the GPU,
are contiguous and 16-byte aligned.  A buffer that a call writes counts as
modified in place: a recorded graph that saved it before refuses to go back.
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch

__all__ = [
    "DGError", "library_path", "load_library",
    "dg_fp8_gemm_nt", "dg_fp8_gemm_nt_acc", "dg_fp8_gemm_grouped_contiguous",
    "dg_fp8_gemm_grouped_masked",
    "dg_quantize_fp8_per_token", "dg_quantize_fp8_per_token_bf16", "dg_quantize_fp8_per_block",
    "dg_fp8_gemm_nt_e8m0", "dg_fp8_gemm_grouped_contiguous_e8m0", "dg_fp8_gemm_grouped_masked_e8m0",
    "dg_quantize_fp8_per_token_e8m0", "dg_quantize_fp8_per_block_e8m0", "e8m0_pitch",
    "dg_status_string",
    "dg_moe_topk", "dg_moe_topk_backward", "dg_moe_mlp_fp8", "dg_moe_mlp_fp8_e8m0",
    "dg_fp8_gemm_nt_lora", "dg_fp8_gemm_nt_lora_e8m0",
    "dg_moe_mlp_fp8_workspace", "dg_fp8_gemm_nt_lora_workspace",
    "dg_moe_sort", "dg_moe_sort_rows", "dg_moe_sort_workspace",
    "dg_moe_dispatch", "dg_moe_dispatch_fp8", "dg_moe_dispatch_fp8_e8m0", "dg_moe_dispatch_int8",
    "dg_moe_unpermute", "dg_moe_unpermute_backward",
    "dg_swiglu", "dg_swiglu_quantize_fp8", "dg_swiglu_quantize_fp8_e8m0", "dg_swiglu_quantize_int8",
    "dg_swiglu_backward",
    "dg_int8_gemm_nt", "dg_int8_gemm_grouped_contiguous", "dg_quantize_int8_per_row",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdgfp8.so")
_lib = None

DG_OK = 0


class DGError(RuntimeError):
    def __init__(self, func: str, status: int):
        self.status = status
        super().__init__(f"{func} failed with status {status}: {dg_status_string(status)}")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libdgfp8.so (built in-tree); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with `python -m fp8_block_scaled_gemm_amd.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    pi64 = ctypes.POINTER(i64)
    for name, args in [
        ("dg_fp8_gemm_nt", [p, p, p, p, p, i64, i64, i64, p]),
        ("dg_fp8_gemm_nt_acc", [p, p, p, p, p, p, i64, i64, i64, p]),
        ("dg_fp8_gemm_grouped_contiguous", [p, p, p, p, p, p, i64, i64, i64, i64, p]),
        ("dg_fp8_gemm_grouped_masked", [p, p, p, p, p, p, i64, i64, i64, i64, p]),
        ("dg_quantize_fp8_per_token", [p, i64, i64, p, p, p]),
        ("dg_quantize_fp8_per_token_bf16", [p, i64, i64, p, p, p]),
        ("dg_quantize_fp8_per_block", [p, i64, i64, p, p, p]),
        ("dg_fp8_gemm_nt_e8m0", [p, p, p, p, p, i64, i64, i64, p]),
        ("dg_fp8_gemm_grouped_contiguous_e8m0", [p, p, p, p, p, p, i64, i64, i64, i64, p]),
        ("dg_fp8_gemm_grouped_masked_e8m0", [p, p, p, p, p, p, i64, i64, i64, i64, p]),
        ("dg_quantize_fp8_per_token_e8m0", [p, i64, i64, p, p, p]),
        ("dg_quantize_fp8_per_block_e8m0", [p, i64, i64, p, p, p]),
        ("dg_moe_topk", [p] * 4 + [i64] * 5 + [i32, i32, f32, p]),
        ("dg_moe_topk_bf16", [p] * 4 + [i64] * 5 + [i32, i32, f32, p]),
        ("dg_moe_topk_backward", [p] * 4 + [i64] * 3 + [i32, i32, f32, p]),
        ("dg_moe_topk_backward_bf16", [p] * 4 + [i64] * 3 + [i32, i32, f32, p]),
        ("dg_moe_mlp_fp8", [p] * 9 + [i64] * 5 + [p, i64, p]),
        ("dg_moe_mlp_fp8_e8m0", [p] * 9 + [i64] * 5 + [p, i64, p]),
        ("dg_moe_mlp_fp8_workspace", [i64] * 5 + [pi64]),
        ("dg_fp8_gemm_nt_lora", [p] * 10 + [i64] * 5 + [p, i64, p]),
        ("dg_fp8_gemm_nt_lora_e8m0", [p] * 10 + [i64] * 5 + [p, i64, p]),
        ("dg_fp8_gemm_nt_lora_workspace", [i64] * 5 + [pi64]),
        ("dg_moe_sort", [p] * 4 + [i64] * 4 + [p, i64, p]),
        ("dg_moe_sort_rows", [i64] * 3 + [pi64]),
        ("dg_moe_sort_workspace", [i64] * 3 + [pi64]),
        ("dg_moe_dispatch", [p] * 6 + [i64] * 5 + [p, i64, p]),
        ("dg_moe_dispatch_fp8", [p] * 7 + [i64] * 5 + [p, i64, p]),
        ("dg_moe_dispatch_fp8_e8m0", [p] * 7 + [i64] * 5 + [p, i64, p]),
        ("dg_moe_dispatch_int8", [p] * 7 + [i64] * 5 + [p, i64, p]),
        ("dg_moe_unpermute", [p] * 4 + [i64] * 4 + [p]),
        ("dg_moe_unpermute_backward", [p] * 7 + [i64] * 4 + [p]),
        ("dg_swiglu", [p] * 3 + [i64] * 2 + [p]),
        ("dg_swiglu_quantize_fp8", [p] * 4 + [i64] * 2 + [p]),
        ("dg_swiglu_quantize_fp8_e8m0", [p] * 4 + [i64] * 2 + [p]),
        ("dg_swiglu_quantize_int8", [p] * 4 + [i64] * 2 + [p]),
        ("dg_swiglu_backward", [p] * 4 + [i64] * 2 + [p]),
        ("dg_int8_gemm_nt", [p] * 5 + [i64] * 3 + [p]),
        ("dg_int8_gemm_grouped_contiguous", [p] * 6 + [i64] * 4 + [p]),
        ("dg_quantize_int8_per_row", [p, i64, i64, p, p, p]),
        ("dg_quantize_int8_per_row_bf16", [p, i64, i64, p, p, p]),
    ]:
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.dg_status_string.argtypes = [ctypes.c_int]
    lib.dg_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def dg_status_string(status: int) -> str:
    return load_library().dg_status_string(int(status)).decode()


def _stream_ptr(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _bytes(t: torch.Tensor, what: str) -> torch.Tensor:
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"{what} must be uint8 or float8_e4m3fn codes, got {t.dtype}")
    return t


def _check(t: torch.Tensor, what: str, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


_D_TYPES = (torch.bfloat16, torch.uint16, torch.int16)


def _device_of(*tensors) -> torch.device:
    """The one device all of a call's tensors live on; a call whose tensors
    span devices is refused (the kernels would read another GPU's memory)."""
    dev = tensors[0].device
    for t in tensors[1:]:
        if t.device != dev:
            raise ValueError(f"all tensors of a call must be on one device, got {dev} and {t.device}")
    return dev


def _call(dev: torch.device, written, name: str, *args):
    # the library launches on the current device, with the stream passed in
    with torch.cuda.device(dev):
        status = getattr(load_library(), name)(*args)
    if status != DG_OK:
        raise DGError(name, status)
    # a recorded graph that saved one of these before refuses to go back with other values
    torch.autograd.graph.increment_version(written)


def dg_fp8_gemm_nt(A, sa, B, sb, D):
    """Dense: D[M][N] = bf16(sum_kb sa[m,kb]*sb[n/128,kb] * A_blk @ B_blk^T)."""
    A, B = _bytes(A, "A"), _bytes(B, "B")
    M, K = A.shape
    N = B.shape[0]
    KB, NB = K // 128, (N + 127) // 128
    _check(A, "A"); _check(B, "B", shape=(N, K))
    _check(sa, "sa", torch.float32, (M, KB)); _check(sb, "sb", torch.float32, (NB, KB))
    _check(D, "D", _D_TYPES, (M, N))
    _call(_device_of(A, sa, B, sb, D), D, "dg_fp8_gemm_nt",
          A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(),
          D.data_ptr(), M, N, K, _stream_ptr(D))
    return D


def dg_fp8_gemm_nt_acc(A, sa, B, sb, C, D):
    """Dense with an fp32 addend: D[M][N] = bf16(C + the dense sum)."""
    A, B = _bytes(A, "A"), _bytes(B, "B")
    M, K = A.shape
    N = B.shape[0]
    KB, NB = K // 128, (N + 127) // 128
    _check(A, "A"); _check(B, "B", shape=(N, K))
    _check(sa, "sa", torch.float32, (M, KB)); _check(sb, "sb", torch.float32, (NB, KB))
    _check(C, "C", torch.float32, (M, N))
    _check(D, "D", _D_TYPES, (M, N))
    _call(_device_of(A, sa, B, sb, C, D), D, "dg_fp8_gemm_nt_acc",
          A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(),
          C.data_ptr(), D.data_ptr(), M, N, K, _stream_ptr(D))
    return D


def dg_fp8_gemm_grouped_contiguous(A, sa, B, sb, D, grouped_layout):
    """Contiguous-grouped: row r of D uses B[grouped_layout[r]]; rows whose
    id is outside [0, G) are not written."""
    A, B = _bytes(A, "A"), _bytes(B, "B")
    M_sum, K = A.shape
    G, N, _ = B.shape
    KB, NB = K // 128, (N + 127) // 128
    _check(A, "A"); _check(B, "B", shape=(G, N, K))
    _check(sa, "sa", torch.float32, (M_sum, KB)); _check(sb, "sb", torch.float32, (G, NB, KB))
    _check(D, "D", _D_TYPES, (M_sum, N))
    _check(grouped_layout, "grouped_layout", torch.int32, (M_sum,))
    _call(_device_of(A, sa, B, sb, D, grouped_layout), D, "dg_fp8_gemm_grouped_contiguous",
          A.data_ptr(), sa.data_ptr(), B.data_ptr(),
          sb.data_ptr(), D.data_ptr(), grouped_layout.data_ptr(), M_sum, N, K, G, _stream_ptr(D))
    return D


def dg_fp8_gemm_grouped_masked(A, sa, B, sb, D, masked_m):
    """Masked-grouped: rows r < masked_m[g] of slab g use B[g]; other rows
    of D are not written."""
    A, B = _bytes(A, "A"), _bytes(B, "B")
    G, M_max, K = A.shape
    _, N, _ = B.shape
    KB, NB = K // 128, (N + 127) // 128
    _check(A, "A"); _check(B, "B", shape=(G, N, K))
    _check(sa, "sa", torch.float32, (G, M_max, KB)); _check(sb, "sb", torch.float32, (G, NB, KB))
    _check(D, "D", _D_TYPES, (G, M_max, N))
    _check(masked_m, "masked_m", torch.int32, (G,))
    _call(_device_of(A, sa, B, sb, D, masked_m), D, "dg_fp8_gemm_grouped_masked",
          A.data_ptr(), sa.data_ptr(), B.data_ptr(),
          sb.data_ptr(), D.data_ptr(), masked_m.data_ptr(), G, M_max, N, K, _stream_ptr(D))
    return D


def dg_quantize_fp8_per_token(x, q=None, s=None):
    """x[M][K] fp32 -> (q[M][K] uint8 e4m3 codes, s[M][K/128] fp32)."""
    _check(x, "x", torch.float32)
    M, K = x.shape
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
    q = _bytes(q, "q")
    _check(q, "q", shape=(M, K)); _check(s, "s", torch.float32, (M, K // 128))
    _call(_device_of(x, q, s), (q, s), "dg_quantize_fp8_per_token",
          x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(),
          _stream_ptr(x))
    return q, s


def dg_quantize_fp8_per_token_bf16(x, q=None, s=None):
    """x[M][K] bf16 -> (q[M][K] uint8 e4m3 codes, s[M][K/128] fp32)."""
    _check(x, "x", torch.bfloat16)
    M, K = x.shape
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
    q = _bytes(q, "q")
    _check(q, "q", shape=(M, K)); _check(s, "s", torch.float32, (M, K // 128))
    _call(_device_of(x, q, s), (q, s), "dg_quantize_fp8_per_token_bf16",
          x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(),
          _stream_ptr(x))
    return q, s


def dg_quantize_fp8_per_block(x, q=None, s=None):
    """x[N][K] fp32 -> (q[N][K] uint8, s[ceil(N/128)][K/128] fp32)."""
    _check(x, "x", torch.float32)
    N, K = x.shape
    NB = (N + 127) // 128
    if q is None:
        q = torch.empty((N, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((NB, K // 128), dtype=torch.float32, device=x.device)
    q = _bytes(q, "q")
    _check(q, "q", shape=(N, K)); _check(s, "s", torch.float32, (NB, K // 128))
    _call(_device_of(x, q, s), (q, s), "dg_quantize_fp8_per_block",
          x.data_ptr(), N, K, q.data_ptr(), s.data_ptr(),
          _stream_ptr(x))
    return q, s


# ------------------------------------------------ power-of-two (E8M0) scales

def e8m0_pitch(kb: int) -> int:
    """Bytes per row of E8M0 scales: K/128 rounded up to a multiple of 4."""
    return (kb + 3) // 4 * 4


def dg_fp8_gemm_nt_e8m0(A, sa, B, sb, D):
    """Dense form with E8M0 scales sa[M][SP], sb[ceil(N/128)][SP] (uint8)."""
    A, B = _bytes(A, "A"), _bytes(B, "B")
    M, K = A.shape
    N = B.shape[0]
    SP, NB = e8m0_pitch(K // 128), (N + 127) // 128
    _check(A, "A"); _check(B, "B", shape=(N, K))
    _check(sa, "sa", torch.uint8, (M, SP)); _check(sb, "sb", torch.uint8, (NB, SP))
    _check(D, "D", _D_TYPES, (M, N))
    _call(_device_of(A, sa, B, sb, D), D, "dg_fp8_gemm_nt_e8m0",
          A.data_ptr(), sa.data_ptr(), B.data_ptr(), sb.data_ptr(),
          D.data_ptr(), M, N, K, _stream_ptr(D))
    return D


def dg_fp8_gemm_grouped_contiguous_e8m0(A, sa, B, sb, D, grouped_layout):
    """Contiguous-grouped form with E8M0 scales sa[M_sum][SP], sb[G][NB][SP]."""
    A, B = _bytes(A, "A"), _bytes(B, "B")
    M_sum, K = A.shape
    G, N, _ = B.shape
    SP, NB = e8m0_pitch(K // 128), (N + 127) // 128
    _check(A, "A"); _check(B, "B", shape=(G, N, K))
    _check(sa, "sa", torch.uint8, (M_sum, SP)); _check(sb, "sb", torch.uint8, (G, NB, SP))
    _check(D, "D", _D_TYPES, (M_sum, N))
    _check(grouped_layout, "grouped_layout", torch.int32, (M_sum,))
    _call(_device_of(A, sa, B, sb, D, grouped_layout), D, "dg_fp8_gemm_grouped_contiguous_e8m0",
          A.data_ptr(), sa.data_ptr(), B.data_ptr(),
          sb.data_ptr(), D.data_ptr(), grouped_layout.data_ptr(), M_sum, N, K, G, _stream_ptr(D))
    return D


def dg_fp8_gemm_grouped_masked_e8m0(A, sa, B, sb, D, masked_m):
    """Masked-grouped form with E8M0 scales sa[G][M_max][SP], sb[G][NB][SP]."""
    A, B = _bytes(A, "A"), _bytes(B, "B")
    G, M_max, K = A.shape
    _, N, _ = B.shape
    SP, NB = e8m0_pitch(K // 128), (N + 127) // 128
    _check(A, "A"); _check(B, "B", shape=(G, N, K))
    _check(sa, "sa", torch.uint8, (G, M_max, SP)); _check(sb, "sb", torch.uint8, (G, NB, SP))
    _check(D, "D", _D_TYPES, (G, M_max, N))
    _check(masked_m, "masked_m", torch.int32, (G,))
    _call(_device_of(A, sa, B, sb, D, masked_m), D, "dg_fp8_gemm_grouped_masked_e8m0",
          A.data_ptr(), sa.data_ptr(), B.data_ptr(),
          sb.data_ptr(), D.data_ptr(), masked_m.data_ptr(), G, M_max, N, K, _stream_ptr(D))
    return D


def dg_quantize_fp8_per_token_e8m0(x, q=None, s=None):
    """x[M][K] fp32 -> (q[M][K] uint8 codes, s[M][SP] uint8 E8M0 exponents).
    A newly allocated s has zero padding bytes; the kernel never writes them."""
    _check(x, "x", torch.float32)
    M, K = x.shape
    SP = e8m0_pitch(K // 128)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.zeros((M, SP), dtype=torch.uint8, device=x.device)
    q = _bytes(q, "q")
    _check(q, "q", shape=(M, K)); _check(s, "s", torch.uint8, (M, SP))
    _call(_device_of(x, q, s), (q, s), "dg_quantize_fp8_per_token_e8m0",
          x.data_ptr(), M, K, q.data_ptr(), s.data_ptr(),
          _stream_ptr(x))
    return q, s


def dg_quantize_fp8_per_block_e8m0(x, q=None, s=None):
    """x[N][K] fp32 -> (q[N][K] uint8, s[ceil(N/128)][SP] uint8 E8M0 exponents)."""
    _check(x, "x", torch.float32)
    N, K = x.shape
    NB, SP = (N + 127) // 128, e8m0_pitch(K // 128)
    if q is None:
        q = torch.empty((N, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.zeros((NB, SP), dtype=torch.uint8, device=x.device)
    q = _bytes(q, "q")
    _check(q, "q", shape=(N, K)); _check(s, "s", torch.uint8, (NB, SP))
    _call(_device_of(x, q, s), (q, s), "dg_quantize_fp8_per_block_e8m0",
          x.data_ptr(), N, K, q.data_ptr(), s.data_ptr(),
          _stream_ptr(x))
    return q, s


# ------------------------------- operators around the products (dg_ops.h)

# Argument checks, allocation and the call itself run in _binding.so
# (csrc/binding.cpp): these operators take microseconds, and checking ten
# tensors in Python took as long as they do.  None of them has a forward-mode
# derivative: a dual tensor's tangent is refused where a new output would lose it.

_SCORING = {"softmax": 0, "sigmoid": 1}
_native = None


def _ops():
    """The compiled binding; raises if it has not been built."""
    global _native
    if _native is None:
        load_library()
        try:
            from . import _binding
        except ImportError as e:
            raise ImportError("the compiled binding is missing or does not load: build it with "
                              "`python -m fp8_block_scaled_gemm_amd.build`") from e
        _native = _binding
    return _native


def _raw_stream(t):
    """torch.cuda.current_stream(t.device).cuda_stream, without its object."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if getattr(t, "is_cuda", False) else 0


def _done(name, result):
    if type(result) is int:
        raise DGError(name, result)
    return result


def _workspace_bytes(name: str, *sizes) -> int:
    out = ctypes.c_int64()
    status = getattr(load_library(), name)(*sizes, ctypes.byref(out))
    if status != DG_OK:
        raise DGError(name, status)
    return out.value


def dg_moe_mlp_fp8_workspace(T, k, E, H, I) -> int:
    """Bytes of a uint8 tensor to pass as ``workspace`` to either form of
    ``dg_moe_mlp_fp8`` with T tokens, k choices, E experts of H x I."""
    return _workspace_bytes("dg_moe_mlp_fp8_workspace", T, k, E, H, I)


def dg_fp8_gemm_nt_lora_workspace(M, N, K, L, R) -> int:
    """Bytes of a uint8 tensor to pass as ``workspace`` to either form of
    ``dg_fp8_gemm_nt_lora`` with M rows, N x K weights, L adapters of rank R."""
    return _workspace_bytes("dg_fp8_gemm_nt_lora_workspace", M, N, K, L, R)


def _score_mode(scoring):
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    return _SCORING[scoring]


def _warn_no_grad(name, where, depth=3):
    warnings.warn(f"{name} records no gradient {where}, though an argument requires one or has a tangent", stacklevel=depth)


class _Topk(torch.autograd.Function):
    """``dg_moe_topk`` with ``dg_moe_topk_backward`` as the gradient of its weights."""

    @staticmethod
    def forward(ctx, logits, k, bias, n_group, topk_group, mode, renormalize, scale):
        ids, weights = _done("dg_moe_topk", _ops().moe_topk(logits, k, None, None, bias, n_group, topk_group, mode,
                                                            renormalize, scale, _raw_stream(logits)))
        ctx.save_for_backward(logits, ids)
        ctx.how = mode, renormalize, scale
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, grad_weights):
        logits, ids = ctx.saved_tensors
        grad = _done("dg_moe_topk_backward", _ops().moe_topk_backward(
            logits, ids, grad_weights.contiguous(), None, *ctx.how, _raw_stream(logits)))
        return (grad,) + (None,) * 7


class _NoGradient(torch.autograd.Function):
    """The output of a call without a backward pass: going back through it is an error."""

    @staticmethod
    def forward(ctx, name, call, *tensors):
        ctx.name = name
        return call()

    @staticmethod
    def backward(ctx, *_):
        raise NotImplementedError(f"{ctx.name} has no gradient: call it under torch.no_grad() or on detached tensors")


def dg_moe_topk(logits, k, ids=None, weights=None, *, bias=None, n_group=1, topk_group=1,
                scoring="softmax", renormalize=True, scale=1.0):
    """Router: logits[T][E] (fp32 or bf16) -> (ids[T][k] int32, weights[T][k]
    fp32), best expert first, -1 and 0 where a row has fewer open experts.
    Where the logits require a gradient, the weights carry it (the bias, which
    only ranks, has none); outputs that the caller gives carry none."""
    mode, renormalize = _score_mode(scoring), bool(renormalize)
    ops = _ops()
    if ops.wants_grad(logits):
        if ids is None and weights is None:
            return _Topk.apply(logits, k, bias, n_group, topk_group, mode, renormalize, scale)
        _warn_no_grad("dg_moe_topk", "in outputs that are given")
    return _done("dg_moe_topk", ops.moe_topk(logits, k, ids, weights, bias, n_group, topk_group, mode, renormalize, scale,
                                             _raw_stream(logits)))


def dg_moe_topk_backward(logits, ids, grad_weights, grad_logits=None, *, scoring="softmax",
                         renormalize=True, scale=1.0):
    """Gradient of ``dg_moe_topk``'s weights with respect to the logits (same
    dtype as the logits), the chosen experts held fixed."""
    return _done("dg_moe_topk_backward", _ops().moe_topk_backward(
        logits, ids, grad_weights, grad_logits, _score_mode(scoring), bool(renormalize), scale, _raw_stream(logits)))


def dg_moe_mlp_fp8(x, sx, ids, weights, w13, s13, w2, s2, y=None, workspace=None):
    """Gated expert layer for up to 256 tokens: y[T][H] bf16 = sum over j of
    weights[t][j] * (quantize(silu(gate) * up) @ w2[e]^T), e = ids[t][j],
    (gate, up) = x @ w13[e]^T; ids outside [0, E) add nothing.  It has no
    backward pass: going back through a new y is an error."""
    ops = _ops()
    if ops.wants_grad(weights, sx, s13, s2):
        return _moe_mlp_no_grad("dg_moe_mlp_fp8", False, x, sx, ids, weights, w13, s13, w2, s2, y, workspace)
    return _done("dg_moe_mlp_fp8", ops.moe_mlp(False, x, sx, ids, weights, w13, s13, w2, s2, y, workspace,
                                               _raw_stream(x)))


def dg_moe_mlp_fp8_e8m0(x, sx, ids, weights, w13, s13, w2, s2, y=None, workspace=None):
    """``dg_moe_mlp_fp8`` with E8M0 scale bytes (rows of ``e8m0_pitch`` bytes)."""
    ops = _ops()
    if ops.wants_grad(weights):
        return _moe_mlp_no_grad("dg_moe_mlp_fp8_e8m0", True, x, sx, ids, weights, w13, s13, w2, s2, y, workspace)
    return _done("dg_moe_mlp_fp8_e8m0", ops.moe_mlp(True, x, sx, ids, weights, w13, s13, w2, s2, y, workspace,
                                                    _raw_stream(x)))


def _moe_mlp_no_grad(name, e8m0, x, sx, ids, weights, w13, s13, w2, s2, y, workspace):
    """The call where an argument requires a gradient: a new y refuses to pass one back."""
    def call():
        return _done(name, _ops().moe_mlp(e8m0, x, sx, ids, weights, w13, s13, w2, s2, y, workspace, _raw_stream(x)))
    if y is None:
        return _NoGradient.apply(name, call, weights, sx, s13, s2)
    _warn_no_grad(name, "in a y that is given", 4)
    return call()


def dg_fp8_gemm_nt_lora(A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, workspace=None):
    """Dense form plus each row's low-rank adapter: D[m] = bf16(dense sum +
    scaling[a] * (x_m @ lora_a[a]^T) @ lora_b[a]^T), a = ids[m], nothing added
    where ids[m] is outside [0, L).  x is the bf16 activation behind A.  No
    gradient is recorded in D."""
    ops = _ops()
    if ops.wants_grad(x, lora_a, lora_b, scaling, sa, sb):
        _warn_no_grad("dg_fp8_gemm_nt_lora", "in D")
    return _done("dg_fp8_gemm_nt_lora", ops.gemm_lora(False, A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling,
                                                      workspace, _raw_stream(A)))


def dg_fp8_gemm_nt_lora_e8m0(A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, workspace=None):
    """``dg_fp8_gemm_nt_lora`` with E8M0 scale bytes for A and B."""
    ops = _ops()
    if ops.wants_grad(x, lora_a, lora_b, scaling):
        _warn_no_grad("dg_fp8_gemm_nt_lora_e8m0", "in D")
    return _done("dg_fp8_gemm_nt_lora_e8m0", ops.gemm_lora(True, A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling,
                                                           workspace, _raw_stream(A)))


# ------- expert layers for many tokens (dg_experts.h), int8 products (dg_int8.h)

_BF16, _FP8, _FP8_E8M0, _INT8 = range(4)  # how rows are held, as in csrc/binding.cpp


def dg_moe_sort_rows(T, k, E) -> int:
    """The most sorted rows that T tokens of k choices among E experts can need
    (a multiple of 128): the rows of the buffers of a dispatch call."""
    return _workspace_bytes("dg_moe_sort_rows", T, k, E)


def dg_moe_sort_workspace(T, k, E) -> int:
    """Bytes of a uint8 tensor to pass as ``workspace`` to ``dg_moe_sort`` or a
    dispatch call."""
    return _workspace_bytes("dg_moe_sort_workspace", T, k, E)


def dg_moe_sort(ids, E, rows=None, layout=None, offsets=None, workspace=None):
    """Tokens sorted by expert: ids[T][k] int32 -> (rows[T][k], layout[M],
    offsets[E + 1]), all int32.  rows holds each pair's sorted row (-1 where the
    id is outside [0, E)), layout each sorted row's expert (-1 for padding: a
    grouped_layout), offsets each expert's first row; every expert's rows are
    padded to 128.  M is ``dg_moe_sort_rows(T, k, E)``, or what a given layout has."""
    return _done("dg_moe_sort", _ops().moe_sort(ids, E, rows, layout, offsets, workspace, _raw_stream(ids)))


class _Dispatch(torch.autograd.Function):
    """``dg_moe_dispatch`` with ``dg_moe_unpermute`` without weights as its gradient."""

    @staticmethod
    def forward(ctx, x, ids, E, workspace):
        out, rows, layout, offsets = _done("dg_moe_dispatch", _ops().moe_dispatch(
            _BF16, x, ids, E, None, None, None, None, None, workspace, _raw_stream(x)))
        ctx.save_for_backward(rows)
        ctx.mark_non_differentiable(rows, layout, offsets)
        return out, rows, layout, offsets

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, *_):
        rows, = ctx.saved_tensors
        grad = grad.contiguous()
        return (_done("dg_moe_unpermute", _ops().moe_unpermute(grad, rows, None, None, _raw_stream(grad))),
                None, None, None)


def dg_moe_dispatch(x, ids, E, out=None, rows=None, layout=None, offsets=None, workspace=None):
    """Sorting and copying in one call: x[T][H] bf16, ids[T][k] -> (out[M][H]
    bf16, rows, layout, offsets), the plan as in ``dg_moe_sort``; rows of padding
    are zeros.  Where x requires a gradient and no buffer is given, out carries it."""
    ops = _ops()
    if ops.wants_grad(x):
        if out is None and rows is None and layout is None and offsets is None:
            return _Dispatch.apply(x, ids, E, workspace)
        _warn_no_grad("dg_moe_dispatch", "in outputs that are given")
    return _done("dg_moe_dispatch", ops.moe_dispatch(_BF16, x, ids, E, out, None, rows, layout, offsets, workspace,
                                                     _raw_stream(x)))


def _no_grad_rows(name, call, x, q, s):
    """A quantizing call whose input requires a gradient: new outputs refuse to
    pass one back, given ones warn, and so do those that are all whole numbers
    (E8M0), which cannot refuse."""
    if q is None and s is None:
        out = _NoGradient.apply(name, call, x)
        if not any(t.requires_grad for t in out):
            _warn_no_grad(name, "in whole numbers", 5)
        return out
    _warn_no_grad(name, "in outputs that are given", 5)
    return call()


def _dispatch_codes(name, held, x, ids, E, q, s, *plan):
    ops = _ops()
    if ops.wants_grad(x):
        return _no_grad_rows(name, lambda: _done(name, ops.moe_dispatch(held, x, ids, E, q, s, *plan, _raw_stream(x))),
                             x, q, s)
    return _done(name, ops.moe_dispatch(held, x, ids, E, q, s, *plan, _raw_stream(x)))


def dg_moe_dispatch_fp8(x, ids, E, q=None, s=None, rows=None, layout=None, offsets=None, workspace=None):
    """``dg_moe_dispatch`` into e4m3 codes, quantized once per token: (q[M][H]
    uint8, s[M][H/128] fp32, rows, layout, offsets); rows of padding in q and s
    are left as they were."""
    return _dispatch_codes("dg_moe_dispatch_fp8", _FP8, x, ids, E, q, s, rows, layout, offsets, workspace)


def dg_moe_dispatch_fp8_e8m0(x, ids, E, q=None, s=None, rows=None, layout=None, offsets=None, workspace=None):
    """``dg_moe_dispatch_fp8`` with E8M0 scale bytes s[M][e8m0_pitch(H/128)]."""
    return _dispatch_codes("dg_moe_dispatch_fp8_e8m0", _FP8_E8M0, x, ids, E, q, s, rows, layout, offsets, workspace)


def dg_moe_dispatch_int8(x, ids, E, q=None, s=None, rows=None, layout=None, offsets=None, workspace=None):
    """``dg_moe_dispatch_fp8`` into int8 with one scale per row: q[M][H] int8, s[M] fp32."""
    return _dispatch_codes("dg_moe_dispatch_int8", _INT8, x, ids, E, q, s, rows, layout, offsets, workspace)


class _Unpermute(torch.autograd.Function):
    """``dg_moe_unpermute`` with its gradients for the rows and the weights."""

    @staticmethod
    def forward(ctx, y, rows, weights, layout):
        out = _done("dg_moe_unpermute", _ops().moe_unpermute(y, rows, weights, None, _raw_stream(y)))
        # the rows themselves are kept only where the weights' gradient needs them
        ctx.rows = y.shape[0]
        ctx.save_for_backward(y if weights is not None and weights.requires_grad else None, rows, weights, layout)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        y, rows, weights, layout = ctx.saved_tensors
        want_y, _, want_weights, _ = ctx.needs_input_grad
        gy, gw = _done("dg_moe_unpermute_backward", _ops().moe_unpermute_backward(
            grad.contiguous(), ctx.rows if y is None else y, rows, weights, layout, None, None, want_y, want_weights,
            _raw_stream(grad)))
        return gy, None, gw, None


def dg_moe_unpermute(y, rows, weights=None, out=None, *, layout=None):
    """Sorted rows back to their tokens: out[T][H] bf16 = sum over j of
    weights[t][j] * y[rows[t][j]] (weights None: ones), entries of rows outside
    [0, M) add nothing.  Where y or the weights require a gradient and no out is
    given, out carries it, for rows that name no row twice; layout is used by
    that gradient alone, which clears only the rows of padding where it is given
    and all of them where it is not.  A given layout belongs to rows: every row
    with an entry of 0 or more is named in rows.  Where pairs were dropped from
    rows after the sort, leave layout out or write -1 into their rows' entries,
    else those rows of y's gradient are not written."""
    ops = _ops()
    if ops.wants_grad(y, weights):
        if out is None:
            return _Unpermute.apply(y, rows, weights, layout)
        _warn_no_grad("dg_moe_unpermute", "in an out that is given")
    return _done("dg_moe_unpermute", ops.moe_unpermute(y, rows, weights, out, _raw_stream(y)))


def dg_moe_unpermute_backward(grad, y, rows, weights=None, layout=None, grad_y=None, grad_weights=None):
    """Gradients of ``dg_moe_unpermute``: grad[T][H] bf16 -> (grad_y[M][H] bf16,
    grad_weights[T][k] fp32, or None where weights is None and none is given).
    Rows of padding are zeros in grad_y where layout is given or grad_y is new;
    a given grad_y keeps them without layout.  No row may be named twice in rows,
    and a given layout belongs to rows as in ``dg_moe_unpermute``: rows with an
    entry of 0 or more that rows does not name are not written."""
    want_weights = weights is not None or grad_weights is not None
    return _done("dg_moe_unpermute_backward", _ops().moe_unpermute_backward(
        grad, y, rows, weights, layout, grad_y, grad_weights, True, want_weights, _raw_stream(y)))


class _Swiglu(torch.autograd.Function):
    """``dg_swiglu`` with ``dg_swiglu_backward`` as its gradient."""

    @staticmethod
    def forward(ctx, z, layout):
        ctx.save_for_backward(z, layout)
        return _done("dg_swiglu", _ops().swiglu(_BF16, z, layout, None, None, _raw_stream(z)))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        z, layout = ctx.saved_tensors
        return _done("dg_swiglu_backward", _ops().swiglu_backward(z, grad.contiguous(), layout, None, _raw_stream(z))), None


def dg_swiglu(z, layout=None, h=None):
    """Gate between an expert's products: z[M][2I] bf16 -> h[M][I] bf16 =
    silu(z[:, :I]) * z[:, I:]; rows whose layout entry is negative are zeros.
    Where z requires a gradient and no h is given, h carries it."""
    ops = _ops()
    if ops.wants_grad(z):
        if h is None:
            return _Swiglu.apply(z, layout)
        _warn_no_grad("dg_swiglu", "in an h that is given")
    return _done("dg_swiglu", ops.swiglu(_BF16, z, layout, h, None, _raw_stream(z)))


def _swiglu_codes(name, held, z, layout, q, s):
    ops = _ops()
    if ops.wants_grad(z):
        return _no_grad_rows(name, lambda: _done(name, ops.swiglu(held, z, layout, q, s, _raw_stream(z))), z, q, s)
    return _done(name, ops.swiglu(held, z, layout, q, s, _raw_stream(z)))


def dg_swiglu_quantize_fp8(z, layout=None, q=None, s=None):
    """``dg_swiglu`` into e4m3 codes without a rounding between: (q[M][I] uint8,
    s[M][I/128] fp32); rows whose layout entry is negative are left as they were."""
    return _swiglu_codes("dg_swiglu_quantize_fp8", _FP8, z, layout, q, s)


def dg_swiglu_quantize_fp8_e8m0(z, layout=None, q=None, s=None):
    """``dg_swiglu_quantize_fp8`` with E8M0 scale bytes s[M][e8m0_pitch(I/128)]."""
    return _swiglu_codes("dg_swiglu_quantize_fp8_e8m0", _FP8_E8M0, z, layout, q, s)


def dg_swiglu_quantize_int8(z, layout=None, q=None, s=None):
    """``dg_swiglu_quantize_fp8`` into int8 with one scale per row: q[M][I] int8, s[M] fp32."""
    return _swiglu_codes("dg_swiglu_quantize_int8", _INT8, z, layout, q, s)


def dg_swiglu_backward(z, grad_h, layout=None, grad_z=None):
    """Gradient of ``dg_swiglu``: (z[M][2I], grad_h[M][I]) bf16 -> grad_z[M][2I]
    bf16; rows whose layout entry is negative are zeros."""
    return _done("dg_swiglu_backward", _ops().swiglu_backward(z, grad_h, layout, grad_z, _raw_stream(z)))


def dg_int8_gemm_nt(A, sa, B, sb, D):
    """Dense int8 product: D[M][N] = bf16(sa[m] * sb[n] * (A @ B^T)), A[M][K] and
    B[N][K] int8, sa[M] and sb[N] fp32, the sums exact.  No gradient is recorded in D."""
    ops = _ops()
    if ops.wants_grad(sa, sb):
        _warn_no_grad("dg_int8_gemm_nt", "in D")
    return _done("dg_int8_gemm_nt", ops.int8_gemm(A, sa, B, sb, D, None, _raw_stream(A)))


def dg_int8_gemm_grouped_contiguous(A, sa, B, sb, D, grouped_layout):
    """Contiguous-grouped int8 product: row r of D uses B[grouped_layout[r]]
    ([G][N][K] int8) and sb[G][N]; rows whose id is outside [0, G) are not
    written.  No gradient is recorded in D."""
    ops = _ops()
    if ops.wants_grad(sa, sb):
        _warn_no_grad("dg_int8_gemm_grouped_contiguous", "in D")
    if grouped_layout is None:
        raise TypeError("grouped_layout must be a torch.Tensor")
    return _done("dg_int8_gemm_grouped_contiguous", ops.int8_gemm(A, sa, B, sb, D, grouped_layout, _raw_stream(A)))


def dg_quantize_int8_per_row(x, q=None, s=None):
    """x[M][K] fp32 or bf16 -> (q[M][K] int8, s[M] fp32): per token for the
    activations, per output channel for the weights."""
    name, ops = "dg_quantize_int8_per_row", _ops()
    if ops.wants_grad(x):
        return _no_grad_rows(name, lambda: _done(name, ops.quantize_int8(x, q, s, _raw_stream(x))), x, q, s)
    return _done(name, ops.quantize_int8(x, q, s, _raw_stream(x)))
