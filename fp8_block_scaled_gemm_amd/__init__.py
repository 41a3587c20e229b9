"""MI355X (gfx950) FP8 block-scaled NT GEMM: thin Python binding.

Every function here has the name of the C-ABI entry point it calls
(include/dg_fp8.h, include/dg_ops.h) and only marshals arguments: it checks torch tensor
dtypes, shapes and devices, passes raw device pointers and the current HIP
stream, and raises ``DGError`` on a nonzero status.  All arithmetic runs in
the HIP kernels of ``libdgfp8.so``; there is no CPU fallback, and importing a
function fails loudly when the library has not been built
(``python -m fp8_block_scaled_gemm_amd.build``).

Tensor conventions: e4m3 codes are ``torch.uint8`` (or
``torch.float8_e4m3fn``, viewed as bytes), scales ``torch.float32``, group
arrays ``torch.int32``, and D is ``torch.bfloat16`` (or ``torch.uint16`` /
``torch.int16`` holding bf16 bit patterns).  All tensors live on the GPU,
are contiguous and 16-byte aligned.
"""
from __future__ import annotations

import ctypes
import functools
import os

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

_SCORING = {"softmax": 0, "sigmoid": 1}


def _ptr(t, what, dtype, shape, dev):
    """The data pointer of a contiguous tensor of this dtype and shape on this
    device, which is a GPU; raises like ``_check`` otherwise.  The common case
    is one comparison each: these calls are a few microseconds long."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _check(t, what, dtype, shape)
    raise ValueError(f"all tensors of a call must be on one device, got {dev} and {t.device}")


def _codes_ptr(t, what, shape, dev):
    if getattr(t, "dtype", None) is torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    return _ptr(t, what, torch.uint8, shape, dev)


def _bf16_ptr(t, what, shape, dev):
    dtype = getattr(t, "dtype", None)
    return _ptr(t, what, dtype if dtype in _D_TYPES else _D_TYPES, shape, dev)


def _dims(t, what, n):
    """Shape of a GPU tensor of n dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{what} must have {n} dimensions, got shape {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    return shape


def _enqueue(dev, name, *args):
    """Call a C entry point on the device's current stream (its last argument)."""
    fn = getattr(_lib or load_library(), name)
    stream = torch._C._cuda_getCurrentRawStream(dev.index)  # torch.cuda.current_stream without its object
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != DG_OK:
        raise DGError(name, status)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, *sizes) -> int:
    out = ctypes.c_int64()
    status = getattr(load_library(), name)(*sizes, ctypes.byref(out))
    if status != DG_OK:
        raise DGError(name, status)
    return out.value


def _workspace(ws, nbytes, dev):
    """The caller's workspace, or a new one from the caching allocator (safe to
    drop once the call is enqueued), with its pointer and bytes."""
    if ws is None:
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    elif ws.dtype is not torch.uint8 or ws.dim() != 1 or ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous one-dimensional uint8 tensor on the call's device")
    return ws, ws.data_ptr(), ws.numel()


def _score_mode(scoring):
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    return _SCORING[scoring]


def dg_moe_topk(logits, k, ids=None, weights=None, *, bias=None, n_group=1, topk_group=1,
                scoring="softmax", renormalize=True, scale=1.0):
    """Router: logits[T][E] (fp32 or bf16) -> (ids[T][k] int32, weights[T][k]
    fp32), best expert first, -1 and 0 where a row has fewer open experts."""
    T, E = _dims(logits, "logits", 2)
    dev, mode = logits.device, _score_mode(scoring)
    name = "dg_moe_topk_bf16" if logits.dtype is torch.bfloat16 else "dg_moe_topk"
    x = _ptr(logits, "logits", torch.bfloat16 if name.endswith("bf16") else torch.float32, (T, E), dev)
    b = None if bias is None else _ptr(bias, "bias", torch.float32, (E,), dev)
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    _enqueue(dev, name, x, b, _ptr(ids, "ids", torch.int32, (T, k), dev),
             _ptr(weights, "weights", torch.float32, (T, k), dev), T, E, k, n_group, topk_group,
             mode, int(renormalize), scale)
    return ids, weights


def dg_moe_topk_backward(logits, ids, grad_weights, grad_logits=None, *, scoring="softmax",
                         renormalize=True, scale=1.0):
    """Gradient of ``dg_moe_topk``'s weights with respect to the logits (same
    dtype as the logits), the chosen experts held fixed."""
    T, E = _dims(logits, "logits", 2)
    k = _dims(ids, "ids", 2)[1]
    dev, mode = logits.device, _score_mode(scoring)
    bf16 = logits.dtype is torch.bfloat16
    dtype = torch.bfloat16 if bf16 else torch.float32
    x = _ptr(logits, "logits", dtype, (T, E), dev)
    if grad_logits is None:
        grad_logits = torch.empty((T, E), dtype=dtype, device=dev)
    _enqueue(dev, "dg_moe_topk_backward_bf16" if bf16 else "dg_moe_topk_backward", x,
             _ptr(ids, "ids", torch.int32, (T, k), dev),
             _ptr(grad_weights, "grad_weights", torch.float32, (T, k), dev),
             _ptr(grad_logits, "grad_logits", dtype, (T, E), dev), T, E, k, mode, int(renormalize), scale)
    return grad_logits


def _moe_mlp(name, e8, x, sx, ids, weights, w13, s13, w2, s2, y, workspace):
    T, H = _dims(x, "x", 2)
    k = _dims(ids, "ids", 2)[1]
    E, _, I = _dims(w2, "w2", 3)
    dev = x.device
    if e8:
        st, kh, ki = torch.uint8, e8m0_pitch(H // 128), e8m0_pitch(I // 128)
    else:
        st, kh, ki = torch.float32, H // 128, I // 128
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    ptrs = (_codes_ptr(x, "x", (T, H), dev), _ptr(sx, "sx", st, (T, kh), dev),
            _ptr(ids, "ids", torch.int32, (T, k), dev), _ptr(weights, "weights", torch.float32, (T, k), dev),
            _codes_ptr(w13, "w13", (E, 2 * I, H), dev), _ptr(s13, "s13", st, (E, (2 * I + 127) // 128, kh), dev),
            _codes_ptr(w2, "w2", (E, H, I), dev), _ptr(s2, "s2", st, (E, (H + 127) // 128, ki), dev),
            _bf16_ptr(y, "y", (T, H), dev))
    ws, at, n = _workspace(workspace, _workspace_bytes("dg_moe_mlp_fp8_workspace", T, k, E, H, I), dev)
    _enqueue(dev, name, *ptrs, T, k, E, H, I, at, n)
    return y


def dg_moe_mlp_fp8(x, sx, ids, weights, w13, s13, w2, s2, y=None, workspace=None):
    """Gated expert layer for up to 256 tokens: y[T][H] bf16 = sum over j of
    weights[t][j] * (quantize(silu(gate) * up) @ w2[e]^T), e = ids[t][j],
    (gate, up) = x @ w13[e]^T; ids outside [0, E) add nothing."""
    return _moe_mlp("dg_moe_mlp_fp8", False, x, sx, ids, weights, w13, s13, w2, s2, y, workspace)


def dg_moe_mlp_fp8_e8m0(x, sx, ids, weights, w13, s13, w2, s2, y=None, workspace=None):
    """``dg_moe_mlp_fp8`` with E8M0 scale bytes (rows of ``e8m0_pitch`` bytes)."""
    return _moe_mlp("dg_moe_mlp_fp8_e8m0", True, x, sx, ids, weights, w13, s13, w2, s2, y, workspace)


def _gemm_lora(name, e8, A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, workspace):
    M, K = _dims(A, "A", 2)
    N = _dims(B, "B", 2)[0]
    L, R, _ = _dims(lora_a, "lora_a", 3)
    dev, NB = A.device, (N + 127) // 128
    st, kb = (torch.uint8, e8m0_pitch(K // 128)) if e8 else (torch.float32, K // 128)
    ptrs = (_codes_ptr(A, "A", (M, K), dev), _ptr(sa, "sa", st, (M, kb), dev),
            _codes_ptr(B, "B", (N, K), dev), _ptr(sb, "sb", st, (NB, kb), dev),
            _bf16_ptr(D, "D", (M, N), dev), _ptr(x, "x", torch.bfloat16, (M, K), dev),
            _ptr(lora_a, "lora_a", torch.bfloat16, (L, R, K), dev),
            _ptr(lora_b, "lora_b", torch.bfloat16, (L, N, R), dev),
            _ptr(ids, "ids", torch.int32, (M,), dev), _ptr(scaling, "scaling", torch.float32, (L,), dev))
    ws, at, n = _workspace(workspace, _workspace_bytes("dg_fp8_gemm_nt_lora_workspace", M, N, K, L, R), dev)
    _enqueue(dev, name, *ptrs, M, N, K, L, R, at, n)
    return D


def dg_fp8_gemm_nt_lora(A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, workspace=None):
    """Dense form plus each row's low-rank adapter: D[m] = bf16(dense sum +
    scaling[a] * (x_m @ lora_a[a]^T) @ lora_b[a]^T), a = ids[m], nothing added
    where ids[m] is outside [0, L).  x is the bf16 activation behind A."""
    return _gemm_lora("dg_fp8_gemm_nt_lora", False, A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling,
                      workspace)


def dg_fp8_gemm_nt_lora_e8m0(A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, workspace=None):
    """``dg_fp8_gemm_nt_lora`` with E8M0 scale bytes for A and B."""
    return _gemm_lora("dg_fp8_gemm_nt_lora_e8m0", True, A, sa, B, sb, D, x, lora_a, lora_b, ids,
                      scaling, workspace)
