"""MI355X (gfx950) FP8 block-scaled NT GEMM: thin Python binding.

Every function here has the name of the C-ABI entry point it calls
(include/dg_fp8.h, include/dg_ops.h) and only marshals arguments: it checks
torch tensor dtypes, shapes and devices, passes raw device pointers and the
current HIP stream, and raises ``DGError`` on a nonzero status.  For the
operators of dg_ops.h a compiled extension, ``_binding.so``, does so.  All
arithmetic runs in the HIP kernels of ``libdgfp8.so``; there is no CPU
fallback, and a call fails loudly when the library has not been built
(``python -m fp8_block_scaled_gemm_amd.build``).

Tensor conventions: e4m3 codes are ``torch.uint8`` (or
``torch.float8_e4m3fn``, viewed as bytes), scales ``torch.float32``, group
arrays ``torch.int32``, and D is ``torch.bfloat16`` (or ``torch.uint16`` /
``torch.int16`` holding bf16 bit patterns).  All tensors live on the GPU,
are contiguous and 16-byte aligned.
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


def _call(dev: torch.device, name: str, *args):
    # the library launches on the current device, with the stream passed in
    with torch.cuda.device(dev):
        status = getattr(load_library(), name)(*args)
    if status != DG_OK:
        raise DGError(name, status)


def dg_fp8_gemm_nt(A, sa, B, sb, D):
    """Dense: D[M][N] = bf16(sum_kb sa[m,kb]*sb[n/128,kb] * A_blk @ B_blk^T)."""
    A, B = _bytes(A, "A"), _bytes(B, "B")
    M, K = A.shape
    N = B.shape[0]
    KB, NB = K // 128, (N + 127) // 128
    _check(A, "A"); _check(B, "B", shape=(N, K))
    _check(sa, "sa", torch.float32, (M, KB)); _check(sb, "sb", torch.float32, (NB, KB))
    _check(D, "D", _D_TYPES, (M, N))
    _call(_device_of(A, sa, B, sb, D), "dg_fp8_gemm_nt",
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
    _call(_device_of(A, sa, B, sb, C, D), "dg_fp8_gemm_nt_acc",
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
    _call(_device_of(A, sa, B, sb, D, grouped_layout), "dg_fp8_gemm_grouped_contiguous",
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
    _call(_device_of(A, sa, B, sb, D, masked_m), "dg_fp8_gemm_grouped_masked",
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
    _call(_device_of(x, q, s), "dg_quantize_fp8_per_token",
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
    _call(_device_of(x, q, s), "dg_quantize_fp8_per_token_bf16",
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
    _call(_device_of(x, q, s), "dg_quantize_fp8_per_block",
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
    _call(_device_of(A, sa, B, sb, D), "dg_fp8_gemm_nt_e8m0",
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
    _call(_device_of(A, sa, B, sb, D, grouped_layout), "dg_fp8_gemm_grouped_contiguous_e8m0",
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
    _call(_device_of(A, sa, B, sb, D, masked_m), "dg_fp8_gemm_grouped_masked_e8m0",
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
    _call(_device_of(x, q, s), "dg_quantize_fp8_per_token_e8m0",
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
    _call(_device_of(x, q, s), "dg_quantize_fp8_per_block_e8m0",
          x.data_ptr(), N, K, q.data_ptr(), s.data_ptr(),
          _stream_ptr(x))
    return q, s


# ------------------------------- operators around the products (dg_ops.h)

# Argument checks, allocation and the call itself run in _binding.so
# (csrc/binding.cpp): these operators take microseconds, and checking ten
# tensors in Python took as long as they do.

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
    warnings.warn(f"{name} records no gradient {where}, though an argument requires one", stacklevel=depth)


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
