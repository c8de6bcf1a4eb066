"""Thin ctypes binding over libgmm.so (the C ABI in include/gmm.h).

Argument marshalling only: every step of the grouped GEMM runs in the CUDA
kernels of libgmm.so.  If the library is missing this module raises; there is
no fallback of any kind.  The functions keep the C names:

    h = gmm_create(num_experts, device)
    gmm_run(h, c, a, a_offsets, b, expert_ids, expert_usage_stats)
    gmm_run_int4(h, c, a, a_offsets, b_packed, b_scales, expert_ids, expert_usage_stats, group_size)
    gmm_query_status(h)            # syncs the stream; returns the code
    gmm_error_string(code)
    gmm_destroy(h)

Tensors are torch CUDA tensors: c/a/b bf16, a_offsets uint32 (or int32 holding
the same bits), expert_ids int32, expert_usage_stats uint32/int32 with at least
2 entries, b_packed int32/uint32 words, b_scales bf16.  `stream` defaults to
torch's current stream on the handle's device.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

GMM_OK = 0
GMM_ERR_INVALID_ARG = -1
GMM_ERR_UNSUPPORTED = -2
GMM_ERR_CUDA = -3
GMM_ERR_DEVICE_TIMEOUT = -4
GMM_ERR_BAD_INPUT = -5
GMM_ERR_NO_DEVICE = -6

EXPORTED = ("gmm_create", "gmm_run", "gmm_run_ex", "gmm_run_int4", "gmm_run_int4_ex", "gmm_matmul_int4",
            "gmm_run_fp8", "gmm_run_planes", "gmm_run_noalloc", "gmm_query_status", "gmm_error_string", "gmm_destroy",
            "gmm_dispatch", "gmm_combine", "gmm_combine_grad", "gmm_quantize_fp4", "gmm_dequantize_fp4", "gmm_run_fp4")

# Activations of the optional epilogue (GMM_ACT_* in gmm.h).
GMM_ACT_NONE = 0
GMM_ACT_RELU = 1
GMM_ACT_SILU = 2
GMM_ACT_GELU_TANH = 3
ACTIVATIONS = {"none": GMM_ACT_NONE, "relu": GMM_ACT_RELU, "silu": GMM_ACT_SILU, "gelu_tanh": GMM_ACT_GELU_TANH}

# Element types of the moved rows (GMM_DTYPE_*) and 4-bit formats (GMM_FP4_*) in gmm.h.
GMM_DTYPE_BF16 = 0
GMM_DTYPE_FP16 = 1
GMM_DTYPE_FP32 = 2
GMM_FP4_NV = 0
GMM_FP4_MX = 1
FP4_FORMATS = {"nvfp4": GMM_FP4_NV, "mxfp4": GMM_FP4_MX}
FP4_BLOCKS = {GMM_FP4_NV: 16, GMM_FP4_MX: 32}


class GmmEpilogue(ctypes.Structure):
    """gmm_epilogue: y = act(acc + bias[e, n]) * row_scale[r] before the bf16 store."""
    _fields_ = [("bias", ctypes.c_void_p), ("row_scale", ctypes.c_void_p), ("activation", ctypes.c_int)]

_lib = None


class GmmError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {gmm_error_string(code)} ({code})")
        self.code = code


def library_path() -> str:
    return _build.LIB_PATH


def load_library(path: str | None = None):
    """Load libgmm.so (raises RuntimeError if it is not built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is not built; call ragged_matmul_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I = ctypes.c_void_p, ctypes.c_int
    lib.gmm_create.argtypes = [ctypes.POINTER(P), I, I]
    lib.gmm_create.restype = I
    lib.gmm_run.argtypes = [P, P, P, P, P, P, P, I, I, I, P]
    lib.gmm_run.restype = I
    lib.gmm_run_int4.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, P]
    lib.gmm_run_int4.restype = I
    EP = ctypes.POINTER(GmmEpilogue)
    lib.gmm_run_ex.argtypes = [P, P, P, P, P, P, P, I, I, I, EP, P]
    lib.gmm_run_ex.restype = I
    lib.gmm_run_int4_ex.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, EP, P]
    lib.gmm_run_int4_ex.restype = I
    lib.gmm_matmul_int4.argtypes = [P, P, P, P, P, I, I, I, I, EP, P]
    lib.gmm_run_planes.restype = I
    lib.gmm_run_planes.argtypes = [P, P, P, P, P, P, P, I, I, I, P, EP, P]
    lib.gmm_run_fp8.restype = I
    lib.gmm_run_fp8.argtypes = [P, P, P, P, P, P, P, I, I, I, P, P, P, EP, P]
    lib.gmm_matmul_int4.restype = I
    lib.gmm_run_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
    lib.gmm_run_noalloc.restype = I
    L = ctypes.c_longlong
    lib.gmm_dispatch.argtypes = [P, P, P, P, P, P, P, L, I, I, I, I, P]
    lib.gmm_dispatch.restype = I
    lib.gmm_combine.argtypes = [P, P, L, P, I, P, P, I, I, I, I, P]
    lib.gmm_combine.restype = I
    lib.gmm_combine_grad.argtypes = [P, P, P, P, L, P, I, P, P, I, I, I, I, P]
    lib.gmm_combine_grad.restype = I
    lib.gmm_quantize_fp4.argtypes = [P, P, P, P, L, I, P, I, P, I, I, I, I, P]
    lib.gmm_quantize_fp4.restype = I
    lib.gmm_dequantize_fp4.argtypes = [P, P, L, P, P, P, I, I, I, I, P]
    lib.gmm_dequantize_fp4.restype = I
    lib.gmm_run_fp4.argtypes = [P, P, P, P, P, P, P, I, I, I, P, P, I, P, P, EP, P]
    lib.gmm_run_fp4.restype = I
    lib.gmm_query_status.argtypes = [P, P]
    lib.gmm_query_status.restype = I
    lib.gmm_error_string.argtypes = [I]
    lib.gmm_error_string.restype = ctypes.c_char_p
    lib.gmm_destroy.argtypes = [P]
    lib.gmm_destroy.restype = I
    if path == library_path():
        _lib = lib
    return lib


def gmm_error_string(code: int) -> str:
    return load_library().gmm_error_string(int(code)).decode()


class Handle:
    """Owns a gmm_handle_t; released by gmm_destroy or at garbage collection."""

    def __init__(self, ptr: int, device: int, num_experts: int):
        self.ptr = ptr
        self.device = device
        self.num_experts = num_experts

    def __del__(self):
        try:
            gmm_destroy(self)
        except Exception:
            pass


def gmm_create(num_experts: int, device: int | None = None) -> Handle:
    import torch
    if device is None:
        device = torch.cuda.current_device()
    h = ctypes.c_void_p()
    rc = load_library().gmm_create(ctypes.byref(h), int(num_experts), int(device))
    if rc != GMM_OK:
        raise GmmError(rc, "gmm_create")
    return Handle(h.value, int(device), int(num_experts))


def gmm_destroy(h: Handle) -> None:
    if h is not None and h.ptr:
        ptr, h.ptr = h.ptr, None
        rc = load_library().gmm_destroy(ptr)
        if rc != GMM_OK:
            raise GmmError(rc, "gmm_destroy")


_raw_stream = None


def stream_handle(device: int, stream=None) -> ctypes.c_void_p:
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            # torch's current stream as an integer; the Stream object that current_stream builds
            # costs more than a kernel launch's own marshalling.
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda d: torch.cuda.current_stream(d).cuda_stream)
        return ctypes.c_void_p(_raw_stream(device))
    return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _check(t, name, dtypes, device, min_numel=0):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must live on cuda:{device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if min_numel and t.numel() < min_numel:
        raise ValueError(f"{name} needs at least {min_numel} elements")
    return ctypes.c_void_p(t.data_ptr())


def _ptr(t, name, dtypes, device, min_numel=0):
    """_check's pointer as an integer; one test for a tensor that passes."""
    try:
        if (t.get_device() == device and t.dtype in dtypes and t.is_contiguous()
                and (not min_numel or t.numel() >= min_numel)):
            return t.data_ptr()
    except AttributeError:
        pass
    return _check(t, name, dtypes, device, min_numel).value


_I32_TYPES = None


def _i32_types():
    global _I32_TYPES
    if _I32_TYPES is None:
        import torch
        _I32_TYPES = (torch.int32,) + ((torch.uint32,) if hasattr(torch, "uint32") else ())
    return _I32_TYPES


def _no_rows(rows, pc, pa):
    """Pointers of c and a: both NULL, the library's call without rows, where one of two empty tensors has none."""
    return (pc, pa) if rows or (pc and pa) else (None, None)


def _routing_args(h, a_offsets, expert_ids, stats):
    G = expert_ids.numel()
    i32 = _i32_types()
    return (_ptr(a_offsets, "a_offsets", i32, h.device, G + 1), _ptr(expert_ids, "expert_ids", i32[:1], h.device),
            _ptr(stats, "expert_usage_stats", i32, h.device, 2), G)


def _epilogue(h: Handle, rows: int, N: int, bias, row_scale, activation) -> GmmEpilogue:
    """Marshal the optional epilogue's operands (checked like the others)."""
    import torch
    act = ACTIVATIONS[activation] if isinstance(activation, str) else int(activation)
    pb = None
    if bias is not None:
        if tuple(bias.shape) != (h.num_experts, N):
            raise ValueError(f"bias must be [E, N] = [{h.num_experts}, {N}], got {tuple(bias.shape)}")
        pb = _check(bias, "bias", (torch.bfloat16,), h.device).value
    ps = None
    if row_scale is not None:
        if row_scale.dim() != 1 or row_scale.numel() < rows:
            raise ValueError(f"row_scale must be 1-D with at least {rows} entries")
        ps = _check(row_scale, "row_scale", (torch.float32,), h.device).value
    return GmmEpilogue(pb, ps, act)


def gmm_run(h: Handle, c, a, a_offsets, b, expert_ids, expert_usage_stats, stream=None,
            check: bool = True) -> int:
    """C[r, :] = A[r, :] @ B[expert_ids[g]].T for rows of active groups (asynchronous)."""
    return gmm_run_ex(h, c, a, a_offsets, b, expert_ids, expert_usage_stats, stream=stream, check=check)


def gmm_run_ex(h: Handle, c, a, a_offsets, b, expert_ids, expert_usage_stats, bias=None, row_scale=None,
               activation=GMM_ACT_NONE, stream=None, check: bool = True) -> int:
    """gmm_run with the optional epilogue y = act(acc + bias[e, n]) * row_scale[r] (asynchronous)."""
    import torch
    if a.dim() != 2 or b.dim() != 3 or c.dim() != 2:
        raise ValueError("a must be [rows, K], b [E, N, K], c [rows, N]")
    E, N, K = b.shape
    if a.shape[1] != K or c.shape[1] != N or c.shape[0] != a.shape[0] or E != h.num_experts:
        raise ValueError(f"shape mismatch: a {tuple(a.shape)}, b {tuple(b.shape)}, c {tuple(c.shape)}, "
                         f"handle E={h.num_experts}")
    bf = (torch.bfloat16,)
    pc, pa = _no_rows(c.shape[0], _check(c, "c", bf, h.device), _check(a, "a", bf, h.device))
    pb = _check(b, "b", bf, h.device)
    po, pi, ps, G = _routing_args(h, a_offsets, expert_ids, expert_usage_stats)
    lib = load_library()
    if bias is None and row_scale is None and not activation:
        rc = lib.gmm_run(h.ptr, pc, pa, po, pb, pi, ps, G, N, K, stream_handle(h.device, stream))
    else:
        epi = _epilogue(h, a.shape[0], N, bias, row_scale, activation)
        rc = lib.gmm_run_ex(h.ptr, pc, pa, po, pb, pi, ps, G, N, K, ctypes.byref(epi),
                            stream_handle(h.device, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_run")
    return rc


def gmm_run_int4(h: Handle, c, a, a_offsets, b_packed, b_scales, expert_ids, expert_usage_stats,
                 group_size: int = 128, stream=None, check: bool = True) -> int:
    """4-bit variant: b_packed [E, N, K/8] 32-bit words, b_scales [E, N, K/group_size] bf16."""
    return gmm_run_int4_ex(h, c, a, a_offsets, b_packed, b_scales, expert_ids, expert_usage_stats,
                           group_size=group_size, stream=stream, check=check)


def gmm_run_int4_ex(h: Handle, c, a, a_offsets, b_packed, b_scales, expert_ids, expert_usage_stats,
                    group_size: int = 128, bias=None, row_scale=None, activation=GMM_ACT_NONE, stream=None,
                    check: bool = True) -> int:
    """gmm_run_int4 with the optional epilogue y = act(acc + bias[e, n]) * row_scale[r]."""
    import torch
    if a.dim() != 2 or b_packed.dim() != 3 or c.dim() != 2 or b_scales.dim() != 3:
        raise ValueError("a must be [rows, K], b_packed [E, N, K/8], b_scales [E, N, K/gs], c [rows, N]")
    E, N, KW = b_packed.shape
    K = KW * 8
    if (a.shape[1] != K or c.shape[1] != N or c.shape[0] != a.shape[0] or E != h.num_experts
            or group_size <= 0 or tuple(b_scales.shape) != (E, N, K // group_size)):
        raise ValueError("shape mismatch between a, b_packed, b_scales, c")
    bf = (torch.bfloat16,)
    pc, pa = _no_rows(c.shape[0], _check(c, "c", bf, h.device), _check(a, "a", bf, h.device))
    pq = _check(b_packed, "b_packed", _i32_types(), h.device)
    psc = _check(b_scales, "b_scales", bf, h.device)
    po, pi, ps, G = _routing_args(h, a_offsets, expert_ids, expert_usage_stats)
    lib = load_library()
    if bias is None and row_scale is None and not activation:
        rc = lib.gmm_run_int4(h.ptr, pc, pa, po, pq, psc, pi, ps, G, N, K, int(group_size),
                              stream_handle(h.device, stream))
    else:
        epi = _epilogue(h, a.shape[0], N, bias, row_scale, activation)
        rc = lib.gmm_run_int4_ex(h.ptr, pc, pa, po, pq, psc, pi, ps, G, N, K, int(group_size), ctypes.byref(epi),
                                 stream_handle(h.device, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_run_int4")
    return rc


def gmm_run_planes(h: Handle, c, a, a_offsets, b, expert_ids, expert_usage_stats, a_plane_splits=(0, 0),
                   bias=None, row_scale=None, activation=GMM_ACT_NONE, stream=None, check: bool = True) -> int:
    """bf16 grouped GEMM with A-plane row offsetting: a holds three planes of a_offsets[G] rows
    ([3 * rows, K] with rows = c.shape[0]); output columns n < s0 read plane 0, n < s0 + s1
    plane 1, the rest plane 2 (s0, s1 multiples of 256); then the optional epilogue."""
    import torch
    if a.dim() != 2 or b.dim() != 3 or c.dim() != 2:
        raise ValueError("a must be [3 * rows, K], b [E, N, K], c [rows, N]")
    E, N, K = b.shape
    s0, s1 = (int(x) for x in a_plane_splits)
    planes = 1 if (s0, s1) == (0, 0) else 3
    if a.shape[1] != K or c.shape[1] != N or a.shape[0] < planes * c.shape[0] or E != h.num_experts:
        raise ValueError(f"shape mismatch: a {tuple(a.shape)} (needs {planes} planes of {c.shape[0]} rows), "
                         f"b {tuple(b.shape)}, c {tuple(c.shape)}, handle E={h.num_experts}")
    bf = (torch.bfloat16,)
    pc, pa = _no_rows(c.shape[0], _check(c, "c", bf, h.device), _check(a, "a", bf, h.device))
    pb = _check(b, "b", bf, h.device)
    po, pi, ps, G = _routing_args(h, a_offsets, expert_ids, expert_usage_stats)
    splits = (ctypes.c_int * 2)(s0, s1)
    epi = None
    if bias is not None or row_scale is not None or activation:
        epi = ctypes.byref(_epilogue(h, c.shape[0], N, bias, row_scale, activation))
    rc = load_library().gmm_run_planes(h.ptr, pc, pa, po, pb, pi, ps, G, N, K, splits, epi,
                                       stream_handle(h.device, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_run_planes")
    return rc


def _fp8_types():
    import torch
    return (torch.uint8,) + ((torch.float8_e4m3fn,) if hasattr(torch, "float8_e4m3fn") else ())


def gmm_run_fp8(h: Handle, c, a, a_offsets, b, expert_ids, expert_usage_stats, input_scale, weight_scale,
                scales_granularity_mnk=(1, 128, None), bias=None, row_scale=None, activation=GMM_ACT_NONE,
                stream=None, check: bool = True) -> int:
    """Block-scaled e4m3 grouped GEMM: a [rows, K] and b [E, N, K] e4m3 (uint8 bit patterns or
    float8_e4m3fn), input_scale fp32 [ceil(rows / gm), ...], weight_scale fp32 [E, ceil(N / gn), ...]
    with (gm, gn, gk) = scales_granularity_mnk (gk None: K); then the optional epilogue."""
    import torch
    if a.dim() != 2 or b.dim() != 3 or c.dim() != 2:
        raise ValueError("a must be [rows, K], b [E, N, K], c [rows, N]")
    E, N, K = b.shape
    rows = a.shape[0]
    if a.shape[1] != K or c.shape[1] != N or c.shape[0] != rows or E != h.num_experts:
        raise ValueError(f"shape mismatch: a {tuple(a.shape)}, b {tuple(b.shape)}, c {tuple(c.shape)}, "
                         f"handle E={h.num_experts}")
    gm, gn, gk = scales_granularity_mnk
    gk = K if gk is None else gk
    gran = (ctypes.c_int * 3)(int(gm), int(gn), int(gk))
    nkb = -(-K // gk) if gk > 0 else 0
    if gm > 0 and input_scale.numel() != -(-rows // gm) * nkb:
        raise ValueError(f"input_scale needs ceil(rows / gm) * ceil(K / gk) = {-(-rows // gm) * nkb} entries")
    if gn > 0 and (weight_scale.shape[0] != E or weight_scale.numel() != E * -(-N // gn) * nkb):
        raise ValueError(f"weight_scale must be [E, ceil(N / gn), ceil(K / gk)] = [{E}, {-(-N // gn)}, {nkb}]")
    pc, pa = _no_rows(rows, _check(c, "c", (torch.bfloat16,), h.device), _check(a, "a", _fp8_types(), h.device))
    pb = _check(b, "b", _fp8_types(), h.device)
    pis = _check(input_scale, "input_scale", (torch.float32,), h.device)
    pws = _check(weight_scale, "weight_scale", (torch.float32,), h.device)
    po, pi, ps, G = _routing_args(h, a_offsets, expert_ids, expert_usage_stats)
    epi = None
    if bias is not None or row_scale is not None or activation:
        epi = ctypes.byref(_epilogue(h, rows, N, bias, row_scale, activation))
    rc = load_library().gmm_run_fp8(h.ptr, pc, pa, po, pb, pi, ps, G, N, K, pis, pws, gran, epi,
                                    stream_handle(h.device, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_run_fp8")
    return rc


def gmm_matmul_int4(h: Handle, c, a, b_packed, b_scales, group_size: int = 128, bias=None, row_scale=None,
                    activation=GMM_ACT_NONE, stream=None, check: bool = True) -> int:
    """Dense 4-bit GEMM C = A . w^T (Modular "multistage_gemm_q"): a [M, K] bf16,
    b_packed [N, K/8] 32-bit words, b_scales [N, K/group_size] bf16, c [M, N] bf16.
    Raises ValueError when an operand is not rank-2, as the page's function does.
    `bias` (if given) is [1, N] bf16: the single expert's row."""
    import torch
    for name, t_ in (("c", c), ("a", a), ("b_packed", b_packed), ("b_scales", b_scales)):
        if t_.dim() != 2:
            raise ValueError(f"{name} must be rank-2, got rank {t_.dim()}")
    M, K = a.shape
    N, KW = b_packed.shape
    if KW * 8 != K or tuple(c.shape) != (M, N) or group_size <= 0 or tuple(b_scales.shape) != (N, K // group_size):
        raise ValueError(f"shape mismatch: a {tuple(a.shape)}, b_packed {tuple(b_packed.shape)}, "
                         f"b_scales {tuple(b_scales.shape)}, c {tuple(c.shape)}")
    bf = (torch.bfloat16,)
    pc = _check(c, "c", bf, h.device)
    pa = _check(a, "a", bf, h.device)
    pq = _check(b_packed, "b_packed", _i32_types(), h.device)
    psc = _check(b_scales, "b_scales", bf, h.device)
    epi = None
    if bias is not None or row_scale is not None or activation:
        pb = None
        if bias is not None:
            if tuple(bias.shape) != (1, N):
                raise ValueError(f"bias must be [1, {N}]")
            pb = _check(bias, "bias", bf, h.device).value
        ps = None
        if row_scale is not None:
            if row_scale.dim() != 1 or row_scale.numel() < M:
                raise ValueError(f"row_scale must be 1-D with at least {M} entries")
            ps = _check(row_scale, "row_scale", (torch.float32,), h.device).value
        act = ACTIVATIONS[activation] if isinstance(activation, str) else int(activation)
        epi = ctypes.byref(GmmEpilogue(pb, ps, act))
    rc = load_library().gmm_matmul_int4(h.ptr, pc, pa, pq, psc, M, N, K, int(group_size), epi,
                                        stream_handle(h.device, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_matmul_int4")
    return rc


# ---------------------------------------------------------------- tokens sorted by expert and back

_ROW_TYPES = _TENSOR = _I32 = _U8 = _F32 = _BF16 = None


def _row_types():
    """torch dtype -> GMM_DTYPE_*; the first call also sets the other types that the calls below test
    for (a statement that imports torch costs each of them as much as a tensor's test)."""
    global _ROW_TYPES, _TENSOR, _I32, _U8, _F32, _BF16
    if _ROW_TYPES is None:
        import torch
        _TENSOR, _I32, _U8 = torch.Tensor, (torch.int32,), (torch.uint8,)
        _F32, _BF16 = (torch.float32,), (torch.bfloat16,)
        _ROW_TYPES = {torch.bfloat16: GMM_DTYPE_BF16, torch.float16: GMM_DTYPE_FP16, torch.float32: GMM_DTYPE_FP32}
    return _ROW_TYPES


def _shaped(t, name, dtypes, device, shape):
    """The pointer of a contiguous tensor of exactly this shape."""
    try:
        if t.shape == shape and t.get_device() == device and t.dtype in dtypes and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    p = _check(t, name, dtypes, device).value
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return p


def _check_strided(t, name, dtypes, device, out=False):
    """A 2-D tensor of contiguous rows, any distance apart (an output's must not overlap):
    its pointer, row stride in elements and shape."""
    if not isinstance(t, _TENSOR):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must live on cuda:{device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {len(shape)}-D")
    rows, width = shape
    if t.is_contiguous():
        return t.data_ptr(), width, shape
    stride = t.stride(0) if rows > 1 else width
    if (width > 1 and t.stride(1) != 1) or (out and stride < width):
        raise ValueError(f"{name} must have contiguous rows{' that do not overlap' if out else ''}, got strides {t.stride()}")
    return t.data_ptr(), stride, shape


def _slots(t, name, device):
    p = _ptr(t, name, _I32, device)
    shape = t.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{name} must be [tokens, top_k]")
    return p, shape


def gmm_dispatch(h: Handle, a_offsets, slot_rows, row_slots, slot_experts, rows=None, tokens=None, stream=None,
                 check: bool = True) -> int:
    """Sort the slots of slot_experts [tokens, top_k] (int32; negative: dropped) by expert, stably:
    writes a_offsets [E + 1], slot_rows [tokens, top_k] and row_slots [tokens * top_k], and, when
    `rows` [tokens * top_k, width] and `tokens` [tokens, width] are given, copies each token to its
    rows (asynchronous).  The gradient of the copy is gmm_combine without weights."""
    types, dev = _row_types(), h.device
    pe, shape = _slots(slot_experts, "slot_experts", dev)
    T, k = shape
    po = _ptr(a_offsets, "a_offsets", _i32_types(), dev, h.num_experts + 1)
    psr = _shaped(slot_rows, "slot_rows", _I32, dev, shape)
    prs = _ptr(row_slots, "row_slots", _I32, dev)
    if row_slots.numel() != T * k:
        raise ValueError(f"row_slots must hold {T * k} entries, got {row_slots.numel()}")
    if (rows is None) != (tokens is None):
        raise ValueError("rows and tokens go together")
    pr = pt = None
    stride, width, dtype = 0, 1, GMM_DTYPE_BF16
    if tokens is not None:
        pt, stride, (n, width) = _check_strided(tokens, "tokens", types, dev)
        if n != T:
            raise ValueError(f"tokens must be [{T}, width], got {tuple(tokens.shape)}")
        element = tokens.dtype
        dtype = types[element]
        pr = _shaped(rows, "rows", (element,), dev, (T * k, width))
    rc = load_library().gmm_dispatch(h.ptr, po, psr, prs, pr, pe, pt, stride, T, k, width, dtype,
                                     stream_handle(h.device, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_dispatch")
    return rc


def gmm_combine(h: Handle, out, rows, slot_rows, weights=None, stream=None, check: bool = True) -> int:
    """out[t] = sum_j weights[t, j] * rows[slot_rows[t, j]] (negative slot_rows: nothing); weights fp32
    [tokens, top_k], None: ones.  out [tokens, width] and rows [num_rows, width] of one dtype."""
    types, dev = _row_types(), h.device
    psr, shape = _slots(slot_rows, "slot_rows", dev)
    T, k = shape
    po, stride, (n, width) = _check_strided(out, "out", types, dev, out=True)
    element = out.dtype
    pr = _ptr(rows, "rows", (element,), dev)
    row_shape = rows.shape
    if len(row_shape) != 2 or n != T or row_shape[1] != width:
        raise ValueError(f"out must be [{T}, width] and rows [num_rows, width], got {tuple(out.shape)} and "
                         f"{tuple(rows.shape)}")
    pw = None if weights is None else _shaped(weights, "weights", _F32, dev, shape)
    rc = load_library().gmm_combine(h.ptr, po, stride, pr, row_shape[0], psr, pw, T, k, width, types[element],
                                    stream_handle(dev, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_combine")
    return rc


def gmm_combine_grad(h: Handle, d_rows, d_weights, d_out, rows, slot_rows, weights=None, stream=None,
                     check: bool = True) -> int:
    """The gradient of gmm_combine: d_rows[slot_rows[t, j]] = weights[t, j] * d_out[t] (rows that no slot
    names stay untouched) and d_weights[t, j] = <d_out[t], rows[slot_rows[t, j]]> in fp32 (None: not
    computed, and `rows` may be None).  The rows that slot_rows names must be distinct, as
    gmm_dispatch's are (not checked): the products of slots that share a row are not summed."""
    types, dev = _row_types(), h.device
    psr, shape = _slots(slot_rows, "slot_rows", dev)
    T, k = shape
    pg, stride, (n, width) = _check_strided(d_out, "d_out", types, dev)
    element = d_out.dtype
    pd = _ptr(d_rows, "d_rows", (element,), dev)
    row_shape = d_rows.shape
    if len(row_shape) != 2 or n != T or row_shape[1] != width:
        raise ValueError(f"d_out must be [{T}, width] and d_rows [num_rows, width], got {tuple(d_out.shape)} and "
                         f"{tuple(d_rows.shape)}")
    pr = None
    if rows is not None:
        pr = _shaped(rows, "rows", (element,), dev, row_shape)
    elif d_weights is not None:
        raise ValueError("d_weights needs rows")
    pw = None if weights is None else _shaped(weights, "weights", _F32, dev, shape)
    pdw = None if d_weights is None else _shaped(d_weights, "d_weights", _F32, dev, shape)
    rc = load_library().gmm_combine_grad(h.ptr, pd, pdw, pg, stride, pr, row_shape[0], psr, pw, T, k, width,
                                         types[element], stream_handle(dev, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_combine_grad")
    return rc


# ---------------------------------------------------------------- 4-bit floating point

def _fp4_format(fmt) -> int:
    f = FP4_FORMATS.get(fmt, fmt)
    if f not in FP4_BLOCKS:
        raise ValueError(f"unknown 4-bit format {fmt!r}: one of {tuple(FP4_FORMATS)}")
    return f


def fp4_scale_pitch(K: int, fmt="nvfp4") -> int:
    """Bytes of a row of block scales (one per 16 or 32 of K, padded to a multiple of 16)."""
    return (K // FP4_BLOCKS[_fp4_format(fmt)] + 15) // 16 * 16


def _check_fp4(packed, scales, names, fmt, rows, K, device):
    """Pointers of packed values [rows, K / 2] and their scales [rows, pitch]."""
    return (_shaped(packed, names[0], _U8, device, (rows, K // 2)),
            _shaped(scales, names[1], _U8, device, (rows, (K // FP4_BLOCKS[fmt] + 15) // 16 * 16)))


def _check_global(t, name, device, numel=1):
    p = _ptr(t, name, _F32, device)
    if t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} value(s), got {t.numel()}")
    return p


def gmm_quantize_fp4(h: Handle, packed, scales, x, fmt="nvfp4", row_slots=None, top_k: int = 1, global_scale=None,
                     stream=None, check: bool = True) -> int:
    """Quantise x [src_rows, K] to e2m1 with block scales: packed uint8 [rows, K / 2], scales uint8
    [rows, fp4_scale_pitch(K, fmt)].  With row_slots (int32 [rows], gmm_dispatch's) row r is quantised
    from x[row_slots[r] // top_k]; a negative entry leaves it untouched."""
    types, dev = _row_types(), h.device
    f = _fp4_format(fmt)
    px, stride, (src_rows, K) = _check_strided(x, "x", types, dev)
    ps, rows = None, src_rows
    if row_slots is not None:
        ps = _ptr(row_slots, "row_slots", _I32, dev)
        rows = row_slots.numel()
    pp, psc = _check_fp4(packed, scales, ("packed", "scales"), f, rows, K, dev)
    pg = None if global_scale is None else _check_global(global_scale, "global_scale", dev)
    rc = load_library().gmm_quantize_fp4(h.ptr, pp, psc, px, stride, src_rows, ps, int(top_k), pg, rows, K,
                                         types[x.dtype], f, stream_handle(dev, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_quantize_fp4")
    return rc


def gmm_dequantize_fp4(h: Handle, y, packed, scales, fmt="nvfp4", global_scale=None, stream=None,
                       check: bool = True) -> int:
    """y [rows, K] (bf16, fp16 or fp32) = the values that packed and scales stand for."""
    types, dev = _row_types(), h.device
    f = _fp4_format(fmt)
    py, stride, (rows, K) = _check_strided(y, "y", types, dev, out=True)
    pp, psc = _check_fp4(packed, scales, ("packed", "scales"), f, rows, K, dev)
    pg = None if global_scale is None else _check_global(global_scale, "global_scale", dev)
    rc = load_library().gmm_dequantize_fp4(h.ptr, py, stride, pp, psc, pg, rows, K, types[y.dtype], f,
                                           stream_handle(h.device, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_dequantize_fp4")
    return rc


def gmm_run_fp4(h: Handle, c, a, a_offsets, b, expert_ids, expert_usage_stats, a_scales, b_scales, fmt="nvfp4",
                a_global=None, b_global=None, bias=None, row_scale=None, activation=GMM_ACT_NONE, stream=None,
                check: bool = True) -> int:
    """Grouped GEMM on microscaled 4-bit operands: a uint8 [rows, K / 2] with a_scales [rows, pitch],
    b uint8 [E, N, K / 2] with b_scales [E, N, pitch] (pitch = fp4_scale_pitch(K, fmt)); a_global one
    fp32 value, b_global fp32 [E]; then the optional epilogue."""
    _row_types()
    f, dev = _fp4_format(fmt), h.device
    pb = _ptr(b, "b", _U8, dev)
    shape = b.shape
    if len(shape) != 3 or shape[0] != h.num_experts:
        raise ValueError(f"b must be [{h.num_experts}, N, K / 2], got {tuple(shape)}")
    E, N, KB = shape
    K = 2 * KB
    pitch = (K // FP4_BLOCKS[f] + 15) // 16 * 16
    if a.dim() != 2:
        raise ValueError(f"a must be [rows, K / 2], got {tuple(a.shape)}")
    rows = a.shape[0]
    pc, pa = _no_rows(rows, _shaped(c, "c", _BF16, dev, (rows, N)), _shaped(a, "a", _U8, dev, (rows, KB)))
    pas = _shaped(a_scales, "a_scales", _U8, dev, (rows, pitch))
    pbs = _shaped(b_scales, "b_scales", _U8, dev, (E, N, pitch))
    pga = None if a_global is None else _check_global(a_global, "a_global", dev)
    pgb = None if b_global is None else _check_global(b_global, "b_global", dev, E)
    po, pi, ps, G = _routing_args(h, a_offsets, expert_ids, expert_usage_stats)
    epi = None
    if bias is not None or row_scale is not None or activation:
        epi = ctypes.byref(_epilogue(h, rows, N, bias, row_scale, activation))
    rc = load_library().gmm_run_fp4(h.ptr, pc, pa, po, pb, pi, ps, G, N, K, pas, pbs, f, pga, pgb, epi,
                                    stream_handle(dev, stream))
    if check and rc != GMM_OK:
        raise GmmError(rc, "gmm_run_fp4")
    return rc


def gmm_query_status(h: Handle, stream=None) -> int:
    return load_library().gmm_query_status(h.ptr, stream_handle(h.device, stream))
