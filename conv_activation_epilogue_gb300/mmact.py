"""Thin Python binding over libmmact.so (the C ABI in include/mmact.h).

Argument marshalling only: every function here checks that the torch tensors
it is handed are CUDA, contiguous and of a supported dtype, turns them into
raw device pointers and sizes, calls the C entry point of the same name and
raises MmactError on a non-OK status.  All arithmetic runs in the library's
CUDA kernels; there is no CPU path.  If the library is not built, the first
call raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libmmact.so")

MMACT_OK, MMACT_ERR_INVALID_ARG, MMACT_ERR_UNSUPPORTED, MMACT_ERR_CUDA, MMACT_ERR_TIMEOUT = range(5)
ACT = {"none": 0, "relu": 1, "leaky_relu": 2, "tanh": 3, "sigmoid": 4, "gelu": 5,
       "silu": 6}   # silu: MXFP4 and 8-bit products and mmact_moe only
DTYPE = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
FP8_DTYPE = {torch.float8_e4m3fn: 5, torch.float8_e5m2: 6}   # codes of 8-bit matrices
MMACT_MXFP4 = 4  # mmact_moe's weights in the 4-bit microscaled format
MMACT_TF32 = 3   # fp32 inputs computed as tf32 (one pass); float32 tensors default to split precision

_lib = None

# Exported C symbols, as declared in include/mmact.h.
SYMBOLS = [
    "mmact_gemm", "mmact_gemm_residual", "mmact_gemm_split", "mmact_gemm_split_noalloc", "mmact_conv2d",
    "mmact_conv2d_split", "mmact_conv2d_residual", "mmact_conv2d_nhwc_residual",
    "mmact_conv2d_nhwc",
    "mmact_conv2d_out_shape", "mmact_conv2d_producer", "mmact_get_last_error",
    "mmact_set_wait_timeout_ns",
    "mmact_selftest_wait_timeout", "mmact_set_gemm_tile_n", "mmact_set_gemm_split_k",
    "mmact_gemm_split_k_choice", "mmact_set_gemm_pair", "mmact_gemm_kernel_choice", "mmact_set_conv_tmem",
    "mmact_gemm_auto", "mmact_gemm_auto_choice", "mmact_conv2d_auto", "mmact_conv2d_auto_choice",
    "mmact_set_gemm_l2_policy", "mmact_tensor_map_cache_stats", "mmact_status_string", "mmact_version",
    "mmact_mxfp4_size", "mmact_quantize_mxfp4", "mmact_dequantize_mxfp4", "mmact_gemm_mxfp4",
    "mmact_linear_mxfp4", "mmact_linear_mxfp4_workspace_bytes", "mmact_moe", "mmact_moe_workspace_bytes",
    "mmact_set_gemm_mxfp4_kernel",
    "mmact_fp8_size", "mmact_quantize_fp8", "mmact_dequantize_fp8", "mmact_gemm_fp8", "mmact_linear_fp8",
    "mmact_linear_fp8_workspace_bytes", "mmact_linear_fp8_backward", "mmact_linear_fp8_backward_workspace_bytes",
    "mmact_set_gemm_fp8_kernel",
    "mmact_moe_route", "mmact_moe_route_workspace_bytes", "mmact_moe_route_backward",
]


class MmactError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load(path: str = LIBRARY) -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"libmmact.so not found at {path}; build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
    L = ctypes.CDLL(path)
    vp, i64, i32, f32, u64, ci = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                                  ctypes.c_uint64, ctypes.c_int)
    p_i32 = ctypes.POINTER(i32)
    L.mmact_gemm.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, f32, vp]
    L.mmact_gemm_residual.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, f32, vp]
    L.mmact_gemm_residual.restype = ci
    L.mmact_gemm_split.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, f32, vp, vp]
    L.mmact_gemm_split_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, f32, vp]
    L.mmact_gemm_split_noalloc.restype = ci
    conv = [vp, vp, vp, vp] + [i64] * 7 + [p_i32, p_i32, p_i32, ci, ci, ci, f32]
    L.mmact_conv2d.argtypes = conv + [vp]
    L.mmact_conv2d_split.argtypes = conv + [vp, vp]
    L.mmact_conv2d_auto.argtypes = conv + [vp, vp]
    L.mmact_conv2d_auto.restype = ci
    L.mmact_conv2d_auto_choice.argtypes = [i64] * 7 + [p_i32, p_i32, p_i32, ci, ci, ci, ctypes.POINTER(ci)]
    L.mmact_conv2d_auto_choice.restype = ci
    L.mmact_gemm_auto.argtypes = [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, f32, vp, vp]
    L.mmact_gemm_auto.restype = ci
    L.mmact_gemm_auto_choice.argtypes = [i64, i64, i64, ci, ci, ci, ctypes.POINTER(ci)]
    L.mmact_gemm_auto_choice.restype = ci
    L.mmact_conv2d_nhwc.argtypes = conv + [vp]
    L.mmact_conv2d_nhwc.restype = ci
    conv_res = [vp, vp, vp, vp, vp] + [i64] * 7 + [p_i32, p_i32, p_i32, ci, ci, ci, f32, vp]
    L.mmact_conv2d_residual.argtypes = conv_res
    L.mmact_conv2d_residual.restype = ci
    L.mmact_conv2d_nhwc_residual.argtypes = conv_res
    L.mmact_conv2d_nhwc_residual.restype = ci
    L.mmact_conv2d_out_shape.argtypes = [i64, i64, i64, i64, p_i32, p_i32, p_i32,
                                         ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.mmact_conv2d_producer.argtypes = [i64] * 7 + [p_i32, p_i32, p_i32, ci, ci]
    L.mmact_conv2d_producer.restype = ci
    L.mmact_get_last_error.argtypes = [vp]
    L.mmact_set_wait_timeout_ns.argtypes = [u64]
    L.mmact_set_wait_timeout_ns.restype = None
    L.mmact_selftest_wait_timeout.argtypes = [u64, vp]
    L.mmact_set_gemm_tile_n.argtypes = [ci]
    L.mmact_set_gemm_split_k.argtypes = [ci]
    L.mmact_set_gemm_pair.argtypes = [ci]
    L.mmact_set_conv_tmem.argtypes = [ci]
    L.mmact_set_gemm_l2_policy.argtypes = [ci]
    L.mmact_set_gemm_l2_policy.restype = ci
    L.mmact_gemm_kernel_choice.argtypes = [i64, i64, i64, ci, ctypes.POINTER(ci)]
    L.mmact_gemm_split_k_choice.argtypes = [i64, i64, i64, ctypes.POINTER(ci)]
    L.mmact_tensor_map_cache_stats.argtypes = [ctypes.POINTER(u64), ctypes.POINTER(u64)]
    L.mmact_tensor_map_cache_stats.restype = ci
    L.mmact_status_string.argtypes = [ci]
    L.mmact_status_string.restype = ctypes.c_char_p
    L.mmact_version.argtypes = []
    p_i64 = ctypes.POINTER(i64)
    L.mmact_mxfp4_size.argtypes = [i64, i64, p_i64, p_i64]
    L.mmact_quantize_mxfp4.argtypes = [vp, vp, vp, i64, i64, ci, ci, vp]
    L.mmact_dequantize_mxfp4.argtypes = [vp, vp, vp, i64, i64, ci, vp]
    L.mmact_gemm_mxfp4.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, f32, vp]
    L.mmact_linear_mxfp4.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, f32, vp, vp]
    L.mmact_linear_mxfp4_workspace_bytes.argtypes = [i64, i64, p_i64]
    L.mmact_moe.argtypes = [vp] * 12 + [i64] * 5 + [ci, ci, ci, f32, ci, ci, vp, vp]
    L.mmact_moe_workspace_bytes.argtypes = [i64] * 5 + [p_i64]
    L.mmact_set_gemm_mxfp4_kernel.argtypes = [ci]
    L.mmact_fp8_size.argtypes = [i64, i64, p_i64, p_i64]
    L.mmact_quantize_fp8.argtypes = [vp, vp, vp, i64, i64, ci, ci, i64, ci, vp]
    L.mmact_dequantize_fp8.argtypes = [vp, vp, vp, i64, i64, ci, ci, vp]
    L.mmact_gemm_fp8.argtypes = [vp] * 6 + [i64, i64, i64, ci, ci, ci, ci, f32, vp]
    L.mmact_linear_fp8.argtypes = [vp] * 5 + [i64, i64, i64, ci, ci, ci, ci, f32, vp, vp]
    L.mmact_linear_fp8_workspace_bytes.argtypes = [i64, i64, p_i64]
    L.mmact_linear_fp8_backward.argtypes = [vp] * 7 + [i64, i64, i64, ci, ci, ci, ci, vp, vp]
    L.mmact_linear_fp8_backward_workspace_bytes.argtypes = [i64, i64, i64, p_i64]
    L.mmact_moe_route.argtypes = [vp] * 6 + [i64, i64, i64, ci, ci, f32, vp, vp]
    L.mmact_moe_route_workspace_bytes.argtypes = [i64, i64, p_i64]
    L.mmact_moe_route_backward.argtypes = [vp] * 7 + [i64, i64, i64, ci, ci, f32, vp]
    L.mmact_set_gemm_fp8_kernel.argtypes = [ci]
    for name in ("mmact_set_gemm_fp8_kernel", "mmact_moe_route", "mmact_moe_route_workspace_bytes", "mmact_moe_route_backward",
                 "mmact_fp8_size", "mmact_quantize_fp8", "mmact_dequantize_fp8", "mmact_gemm_fp8", "mmact_linear_fp8",
                 "mmact_linear_fp8_workspace_bytes", "mmact_linear_fp8_backward",
                 "mmact_linear_fp8_backward_workspace_bytes"):
        getattr(L, name).restype = ci
    for name in ("mmact_mxfp4_size", "mmact_quantize_mxfp4", "mmact_dequantize_mxfp4", "mmact_gemm_mxfp4",
                 "mmact_linear_mxfp4", "mmact_linear_mxfp4_workspace_bytes", "mmact_moe",
                 "mmact_moe_workspace_bytes", "mmact_set_gemm_mxfp4_kernel"):
        getattr(L, name).restype = ci
    for name in ("mmact_gemm", "mmact_gemm_split", "mmact_conv2d", "mmact_conv2d_split",
                 "mmact_conv2d_out_shape", "mmact_get_last_error", "mmact_selftest_wait_timeout",
                 "mmact_set_gemm_tile_n", "mmact_set_gemm_split_k", "mmact_gemm_split_k_choice",
                 "mmact_set_gemm_pair", "mmact_gemm_kernel_choice", "mmact_set_conv_tmem",
                 "mmact_version"):
        getattr(L, name).restype = ci
    _lib = L
    return L


def status_string(status: int) -> str:
    return load().mmact_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != MMACT_OK:
        raise MmactError(status, where)


# the current stream's raw handle without building a torch.cuda.Stream object
# (a few microseconds per call on small launches); torch's public route otherwise
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_CUR_DEVICE = getattr(torch._C, "_cuda_getDevice", None)


def _stream_handle(stream) -> int | None:
    if stream is None:
        if _RAW_STREAM is not None and _CUR_DEVICE is not None:
            return _RAW_STREAM(_CUR_DEVICE()) or None
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _dev(t: torch.Tensor, name: str, dtypes) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} dtype {t.dtype} not in {dtypes}")
    return t.data_ptr()


_IN = (torch.float16, torch.bfloat16, torch.float32)   # float32 inputs: split precision
_OUT = (torch.float16, torch.bfloat16, torch.float32)


def _bias_ptr(bias, n: int):
    if bias is None:
        return None
    _dev(bias, "bias", (torch.float32,))
    if bias.numel() != n:
        raise ValueError(f"bias must have {n} elements")
    return bias.data_ptr()


def _gemm_args(A, B, bias, C):
    pa = _dev(A, "A", _IN)
    pb = _dev(B, "B", _IN)
    pc = _dev(C, "C", _OUT)
    if A.dim() != 2 or B.dim() != 2 or C.dim() != 2:
        raise ValueError("A, B, C must be 2-D")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N) or B.dtype != A.dtype:
        raise ValueError("shape/dtype mismatch: A [M,K], B [K,N], C [M,N], A and B same dtype")
    return pa, pb, _bias_ptr(bias, N), pc, M, N, K


def mmact_gemm(A, B, bias, C, act: str = "none", alpha: float = 0.0, stream=None) -> None:
    """C = act(A @ B + bias) in one fused kernel (see include/mmact.h)."""
    L = load()
    pa, pb, pbias, pc, M, N, K = _gemm_args(A, B, bias, C)
    _check(L.mmact_gemm(pa, pb, pbias, pc, M, N, K, DTYPE[A.dtype], DTYPE[C.dtype], ACT[act],
                        float(alpha), _stream_handle(stream)), "mmact_gemm")


def mmact_gemm_residual(A, B, bias, R, C, act: str = "none", alpha: float = 0.0, stream=None) -> None:
    """C = act(A @ B + bias + R) in one fused kernel; R [M,N] has C's dtype and
    may be C itself (see include/mmact.h)."""
    L = load()
    pa, pb, pbias, pc, M, N, K = _gemm_args(A, B, bias, C)
    pr = _dev(R, "R", _OUT)
    if tuple(R.shape) != (M, N) or R.dtype != C.dtype:
        raise ValueError("R must be [M,N] with C's dtype")
    _check(L.mmact_gemm_residual(pa, pb, pbias, pr, pc, M, N, K, DTYPE[A.dtype], DTYPE[C.dtype],
                                 ACT[act], float(alpha), _stream_handle(stream)), "mmact_gemm_residual")


def mmact_gemm_split(A, B, bias, C, workspace, act: str = "none", alpha: float = 0.0,
                     stream=None) -> None:
    """Two-kernel ablation: workspace (fp32 [M,N]) = A @ B + bias, then C = act(workspace)."""
    L = load()
    pa, pb, pbias, pc, M, N, K = _gemm_args(A, B, bias, C)
    pw = _dev(workspace, "workspace", (torch.float32,))
    if workspace.numel() < M * N:
        raise ValueError("workspace must hold M*N fp32 elements")
    _check(L.mmact_gemm_split(pa, pb, pbias, pc, M, N, K, DTYPE[A.dtype], DTYPE[C.dtype], ACT[act],
                              float(alpha), pw, _stream_handle(stream)), "mmact_gemm_split")


def mmact_gemm_auto(A, B, bias, C, act: str = "none", alpha: float = 0.0, workspace=None, stream=None) -> None:
    """Fused or two-kernel GEMM, decided per shape (see include/mmact.h); the split path
    needs `workspace` (fp32, at least M*N elements) and is never taken without one."""
    L = load()
    pa, pb, pbias, pc, M, N, K = _gemm_args(A, B, bias, C)
    pw = None
    if workspace is not None:
        pw = _dev(workspace, "workspace", (torch.float32,))
        if workspace.numel() < M * N:
            raise ValueError("workspace must hold M*N fp32 elements")
    _check(L.mmact_gemm_auto(pa, pb, pbias, pc, M, N, K, DTYPE[A.dtype], DTYPE[C.dtype], ACT[act],
                             float(alpha), pw, _stream_handle(stream)), "mmact_gemm_auto")


def mmact_gemm_auto_choice(M, N, K, ab_dtype, c_dtype, act: str) -> str:
    """"split" or "fused": the path mmact_gemm_auto takes with a workspace (dtypes: torch dtypes)."""
    out = ctypes.c_int(-1)
    _check(load().mmact_gemm_auto_choice(int(M), int(N), int(K), DTYPE[ab_dtype], DTYPE[c_dtype], ACT[act],
                                         ctypes.byref(out)), "mmact_gemm_auto_choice")
    return "split" if out.value == 1 else "fused"


NOALLOC_MAX_ELEMENTS = 4194304   # MMACT_NOALLOC_MAX_ELEMENTS in include/mmact.h


def mmact_gemm_split_noalloc(A, B, bias, C, act: str = "none", alpha: float = 0.0,
                             stream=None) -> None:
    """mmact_gemm_split using the library's built-in scratch array instead of a
    caller-provided workspace (for callers that cannot allocate; M*N is limited)."""
    L = load()
    pa, pb, pbias, pc, M, N, K = _gemm_args(A, B, bias, C)
    _check(L.mmact_gemm_split_noalloc(pa, pb, pbias, pc, M, N, K, DTYPE[A.dtype], DTYPE[C.dtype],
                                      ACT[act], float(alpha), _stream_handle(stream)),
           "mmact_gemm_split_noalloc")


# ctypes int32 arrays for strides / pads / dilations, kept per value tuple: a call
# site that repeats its geometry reuses them (the library only reads them during
# the call)
_I32_ARRAYS: dict = {}


def _i32(vals, n):
    vals = tuple(int(v) for v in vals)
    if len(vals) != n:
        raise ValueError(f"expected {n} values")
    arr = _I32_ARRAYS.get(vals)
    if arr is None:
        if len(_I32_ARRAYS) > 1024:
            _I32_ARRAYS.clear()
        arr = _I32_ARRAYS[vals] = (ctypes.c_int32 * n)(*vals)
    return arr


_OUT_SHAPES: dict = {}


def mmact_conv2d_out_shape(H, W, kh, kw, stride, pads, dilation) -> tuple:
    """(Ho, Wo) from the library's output-size rule (answers kept per geometry)."""
    key = (int(H), int(W), int(kh), int(kw), tuple(stride), tuple(pads), tuple(dilation))
    hit = _OUT_SHAPES.get(key)
    if hit is not None:
        return hit
    L = load()
    ho, wo = ctypes.c_int64(), ctypes.c_int64()
    _check(L.mmact_conv2d_out_shape(H, W, kh, kw, _i32(stride, 2), _i32(pads, 4),
                                    _i32(dilation, 2), ctypes.byref(ho), ctypes.byref(wo)),
           "mmact_conv2d_out_shape")
    if len(_OUT_SHAPES) > 1024:
        _OUT_SHAPES.clear()
    _OUT_SHAPES[key] = (ho.value, wo.value)
    return ho.value, wo.value


CONV_PRODUCER = {0: "gather", 1: "vector", 2: "window", 3: "tmem"}


def mmact_conv2d_producer(N, C, H, W, Co, kh, kw, stride, pads, dilation, in_dtype, out_dtype) -> str:
    """Which B-tile producer mmact_conv2d uses for this NCHW geometry (a name
    from CONV_PRODUCER); dtypes are torch dtypes."""
    r = load().mmact_conv2d_producer(N, C, H, W, Co, kh, kw, _i32(stride, 2), _i32(pads, 4),
                                     _i32(dilation, 2), DTYPE[in_dtype], DTYPE[out_dtype])
    if r not in CONV_PRODUCER:
        raise ValueError("mmact_conv2d_producer: invalid arguments")
    return CONV_PRODUCER[r]


def _conv_args(x, w, bias, y, stride, pads, dilation):
    px = _dev(x, "x", _IN)
    pw = _dev(w, "w", _IN)
    py = _dev(y, "y", _OUT)
    if x.dim() != 4 or w.dim() != 4 or y.dim() != 4:
        raise ValueError("x, w, y must be 4-D (NCHW / [Co,C,kh,kw])")
    N, C, H, W = x.shape
    Co, C2, kh, kw = w.shape
    if C2 != C or w.dtype != x.dtype:
        raise ValueError("w must be [Co, C, kh, kw] with x's dtype")
    Ho, Wo = mmact_conv2d_out_shape(H, W, kh, kw, stride, pads, dilation)
    if tuple(y.shape) != (N, Co, Ho, Wo):
        raise ValueError(f"y must be {(N, Co, Ho, Wo)}")
    return (px, pw, _bias_ptr(bias, Co), py, N, C, H, W, Co, kh, kw, _i32(stride, 2),
            _i32(pads, 4), _i32(dilation, 2))


def mmact_conv2d(x, w, bias, y, stride=(1, 1), pads=(0, 0, 0, 0), dilation=(1, 1),
                 act: str = "tanh", alpha: float = 0.0, stream=None) -> None:
    """y = act(conv2d(x, w) + bias), NCHW, pads = (top, bottom, left, right)."""
    L = load()
    args = _conv_args(x, w, bias, y, stride, pads, dilation)
    _check(L.mmact_conv2d(*args, DTYPE[x.dtype], DTYPE[y.dtype], ACT[act], float(alpha),
                          _stream_handle(stream)), "mmact_conv2d")


def _residual_ptr(R, y):
    pr = _dev(R, "R", _OUT)
    if tuple(R.shape) != tuple(y.shape) or R.dtype != y.dtype:
        raise ValueError("R must have y's shape and dtype")
    return pr


def mmact_conv2d_residual(x, w, bias, R, y, stride=(1, 1), pads=(0, 0, 0, 0), dilation=(1, 1),
                          act: str = "tanh", alpha: float = 0.0, stream=None) -> None:
    """y = act(conv2d(x, w) + bias + R), NCHW; R has y's shape and dtype and may be y."""
    L = load()
    px, pw, pb, py, *rest = _conv_args(x, w, bias, y, stride, pads, dilation)
    pr = _residual_ptr(R, y)
    _check(L.mmact_conv2d_residual(px, pw, pb, pr, py, *rest, DTYPE[x.dtype], DTYPE[y.dtype], ACT[act],
                                   float(alpha), _stream_handle(stream)), "mmact_conv2d_residual")


def mmact_conv2d_split(x, w, bias, y, workspace, stride=(1, 1), pads=(0, 0, 0, 0),
                       dilation=(1, 1), act: str = "tanh", alpha: float = 0.0, stream=None) -> None:
    """Two-kernel ablation of mmact_conv2d through an fp32 workspace shaped like y."""
    L = load()
    args = _conv_args(x, w, bias, y, stride, pads, dilation)
    pws = _dev(workspace, "workspace", (torch.float32,))
    if workspace.numel() < y.numel():
        raise ValueError("workspace must hold y.numel() fp32 elements")
    _check(L.mmact_conv2d_split(*args, DTYPE[x.dtype], DTYPE[y.dtype], ACT[act], float(alpha), pws,
                                _stream_handle(stream)), "mmact_conv2d_split")


def _in_code(x, tf32: bool) -> int:
    if tf32:
        if x.dtype != torch.float32:
            raise ValueError("tf32=True needs float32 x and w")
        return MMACT_TF32
    return DTYPE[x.dtype]


def mmact_conv2d_auto(x, w, bias, y, stride=(1, 1), pads=(0, 0, 0, 0), dilation=(1, 1),
                      act: str = "tanh", alpha: float = 0.0, workspace=None, stream=None) -> None:
    """NCHW fused or two-kernel conv, decided per geometry (see include/mmact.h)."""
    L = load()
    args = _conv_args(x, w, bias, y, stride, pads, dilation)
    pws = None
    if workspace is not None:
        pws = _dev(workspace, "workspace", (torch.float32,))
        if workspace.numel() < y.numel():
            raise ValueError("workspace must hold y.numel() fp32 elements")
    _check(L.mmact_conv2d_auto(*args, DTYPE[x.dtype], DTYPE[y.dtype], ACT[act], float(alpha), pws,
                               _stream_handle(stream)), "mmact_conv2d_auto")


def mmact_conv2d_auto_choice(N, C, H, W, Co, kh, kw, stride, pads, dilation, in_dtype, out_dtype,
                             act: str) -> str:
    """"split" or "fused": the path mmact_conv2d_auto takes with a workspace."""
    out = ctypes.c_int(-1)
    _check(load().mmact_conv2d_auto_choice(N, C, H, W, Co, kh, kw, _i32(stride, 2), _i32(pads, 4),
                                           _i32(dilation, 2), DTYPE[in_dtype], DTYPE[out_dtype], ACT[act],
                                           ctypes.byref(out)), "mmact_conv2d_auto_choice")
    return "split" if out.value == 1 else "fused"


def mmact_conv2d_nhwc(x, w, bias, y, stride=(1, 1), pads=(0, 0, 0, 0), dilation=(1, 1),
                      act: str = "tanh", alpha: float = 0.0, stream=None, tf32: bool = False) -> None:
    """Channels-last y = act(conv2d(x, w) + bias): x [N,H,W,C], w [Co,kh,kw,C], y [N,Ho,Wo,Co].
    float32 x and w run in split precision (fp32 accuracy), or as tf32 (one pass) with
    tf32=True (see include/mmact.h)."""
    L = load()
    px, pw, pb, py, *rest = _nhwc_args(x, w, bias, y, stride, pads, dilation)
    _check(L.mmact_conv2d_nhwc(px, pw, pb, py, *rest, _in_code(x, tf32), DTYPE[y.dtype], ACT[act],
                               float(alpha), _stream_handle(stream)), "mmact_conv2d_nhwc")


def _nhwc_args(x, w, bias, y, stride, pads, dilation):
    px = _dev(x, "x", _OUT)
    pw = _dev(w, "w", _OUT)
    py = _dev(y, "y", _OUT)
    if x.dim() != 4 or w.dim() != 4 or y.dim() != 4:
        raise ValueError("x, w, y must be 4-D (NHWC / [Co,kh,kw,C] / NHWC)")
    N, H, W, C = x.shape
    Co, kh, kw, C2 = w.shape
    if C2 != C or w.dtype != x.dtype:
        raise ValueError("w must be [Co, kh, kw, C] with x's dtype")
    Ho, Wo = mmact_conv2d_out_shape(H, W, kh, kw, stride, pads, dilation)
    if tuple(y.shape) != (N, Ho, Wo, Co):
        raise ValueError(f"y must be {(N, Ho, Wo, Co)}")
    return (px, pw, _bias_ptr(bias, Co), py, N, C, H, W, Co, kh, kw, _i32(stride, 2), _i32(pads, 4),
            _i32(dilation, 2))


def mmact_conv2d_nhwc_residual(x, w, bias, R, y, stride=(1, 1), pads=(0, 0, 0, 0), dilation=(1, 1),
                               act: str = "tanh", alpha: float = 0.0, stream=None, tf32: bool = False) -> None:
    """Channels-last y = act(conv2d(x, w) + bias + R); R has y's shape [N,Ho,Wo,Co] and dtype."""
    L = load()
    px, pw, pb, py, *rest = _nhwc_args(x, w, bias, y, stride, pads, dilation)
    pr = _residual_ptr(R, y)
    _check(L.mmact_conv2d_nhwc_residual(px, pw, pb, pr, py, *rest, _in_code(x, tf32), DTYPE[y.dtype],
                                        ACT[act], float(alpha), _stream_handle(stream)),
           "mmact_conv2d_nhwc_residual")


_BYTES = (torch.uint8,)


def mmact_mxfp4_size(rows: int, K: int) -> tuple[int, int]:
    """(bytes of codes, bytes of scales) of an MXFP4 matrix [rows, K] (see include/mmact.h)."""
    c, s = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(load().mmact_mxfp4_size(int(rows), int(K), ctypes.byref(c), ctypes.byref(s)), "mmact_mxfp4_size")
    return c.value, s.value


def _mxfp4_ptrs(codes, scales, rows: int, K: int, name: str):
    # the sizes of mmact_mxfp4_size; _dev says what else is wrong
    if not (codes.dtype is torch.uint8 and scales.dtype is torch.uint8 and codes.is_cuda and scales.is_cuda
            and codes.is_contiguous() and scales.is_contiguous()):
        _dev(codes, name + " codes", _BYTES)
        _dev(scales, name + " scales", _BYTES)
    if codes.numel() != rows * ((K + 31) // 32 * 16):
        raise ValueError(f"{name} codes must hold {rows} x {(K + 31) // 32 * 16} bytes")
    if scales.numel() != (rows + 127) // 128 * ((K + 127) // 128) * 512:
        raise ValueError(f"{name} scales must hold {(rows + 127) // 128} x {(K + 127) // 128} tiles of 512 bytes")
    return codes.data_ptr(), scales.data_ptr()


def _matrix(t, name: str):
    """(pointer, dtype code, rows, columns) of a contiguous 2-D CUDA tensor of floats."""
    code = DTYPE.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None or not t.is_cuda or not t.is_contiguous():
        _dev(t, name, _IN)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    return t.data_ptr(), code, rows, cols


def mmact_quantize_mxfp4(x, codes, scales, transposed: bool = False, stream=None) -> None:
    """Quantise x [rows, K] (or, transposed, [K, rows]) to MXFP4 with blocks along K; codes and
    scales are uint8 tensors of mmact_mxfp4_size(rows, K) bytes."""
    px, dt, rows, K = _matrix(x, "x")
    if transposed:
        rows, K = K, rows
    pc, ps = _mxfp4_ptrs(codes, scales, rows, K, "x")
    s = (_lib or load()).mmact_quantize_mxfp4(px, pc, ps, rows, K, dt, 1 if transposed else 0, _stream_handle(stream))
    if s:
        _check(s, "mmact_quantize_mxfp4")


def mmact_dequantize_mxfp4(codes, scales, y, stream=None) -> None:
    """y [rows, K] = the values of an MXFP4 matrix."""
    py, dt, rows, K = _matrix(y, "y")
    pc, ps = _mxfp4_ptrs(codes, scales, rows, K, "y")
    s = (_lib or load()).mmact_dequantize_mxfp4(pc, ps, py, rows, K, dt, _stream_handle(stream))
    if s:
        _check(s, "mmact_dequantize_mxfp4")


def mmact_gemm_mxfp4(a_codes, a_scales, b_codes, b_scales, bias, C, K: int, act: str = "none",
                     alpha: float = 0.0, stream=None) -> None:
    """C = act(A @ B.T + bias) of MXFP4 matrices A [M, K] and B [N, K]; C [M, N]."""
    pc, dt, M, N = _matrix(C, "C")
    pa, psa = _mxfp4_ptrs(a_codes, a_scales, M, K, "A")
    pb, psb = _mxfp4_ptrs(b_codes, b_scales, N, K, "B")
    s = (_lib or load()).mmact_gemm_mxfp4(pa, psa, pb, psb, _bias_ptr(bias, N), pc, M, N, K, dt, ACT[act], alpha,
                                          _stream_handle(stream))
    if s:
        _check(s, "mmact_gemm_mxfp4")


def mmact_linear_mxfp4_workspace_bytes(M: int, K: int) -> int:
    """Bytes of the workspace that mmact_linear_mxfp4 needs for x [M, K]."""
    out = ctypes.c_int64(0)
    _check(load().mmact_linear_mxfp4_workspace_bytes(int(M), int(K), ctypes.byref(out)),
           "mmact_linear_mxfp4_workspace_bytes")
    return out.value


def mmact_linear_mxfp4(x, w_codes, w_scales, bias, C, workspace, act: str = "none", alpha: float = 0.0,
                       stream=None) -> None:
    """C = act(q(x) @ W.T + bias): x [M, K] is quantised to MXFP4 on the way in, W [N, K] is MXFP4."""
    px, xd, M, K = _matrix(x, "x")
    pc, cd, rows, N = _matrix(C, "C")
    if rows != M:
        raise ValueError("x must be [M, K] and C [M, N]")
    pw, ps = _mxfp4_ptrs(w_codes, w_scales, N, K, "W")
    pws = _dev(workspace, "workspace", _BYTES)
    if workspace.numel() < -(-M * ((K + 31) // 32 * 16) // 512) * 512 + (M + 127) // 128 * ((K + 127) // 128) * 512:
        raise ValueError("workspace must hold mmact_linear_mxfp4_workspace_bytes(M, K) bytes")
    s = (_lib or load()).mmact_linear_mxfp4(px, pw, ps, _bias_ptr(bias, N), pc, M, N, K, xd, cd, ACT[act], alpha, pws,
                                            _stream_handle(stream))
    if s:
        _check(s, "mmact_linear_mxfp4")


def mmact_set_gemm_mxfp4_kernel(mode: int) -> None:
    """MXFP4 products: 0 kernel chosen per shape; 1 few rows or tiles; 2 CTA pairs."""
    _check(load().mmact_set_gemm_mxfp4_kernel(int(mode)), "mmact_set_gemm_mxfp4_kernel")


def mmact_fp8_size(rows: int, K: int) -> tuple[int, int]:
    """(bytes of codes, bytes of scales) of an 8-bit matrix [rows, K] (see include/mmact.h)."""
    c, s = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(load().mmact_fp8_size(int(rows), int(K), ctypes.byref(c), ctypes.byref(s)), "mmact_fp8_size")
    return c.value, s.value


_F8 = (torch.float8_e4m3fn, torch.float8_e5m2)


def _device(first, name: str) -> int:
    """The current device, asked for when a call's first tensor lies on any."""
    if not isinstance(first, torch.Tensor) or first.get_device() < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return _CUR_DEVICE() if _CUR_DEVICE is not None else torch.cuda.current_device()


def _on(t, name: str, dtype, dev: int) -> int:
    """Pointer of a contiguous tensor of that dtype on device `dev`, the current one (its stream gets the
    kernels): one line for what is right, as small calls take no longer than their checks."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _dev(t, name, (dtype,))
    raise ValueError(f"{name} is on device {t.get_device()}, the current one is {dev}")


def _matrix_on(t, name: str, dev: int):
    """(pointer, dtype code, rows, columns) of a contiguous 2-D tensor of floats on device `dev`."""
    p, code, rows, cols = _matrix(t, name)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the current one is {dev}")
    return p, code, rows, cols


def _bias_on(bias, n: int, dev: int):
    if bias is None:
        return None
    p = _on(bias, "bias", torch.float32, dev)
    if bias.numel() != n:
        raise ValueError(f"bias must have {n} elements")
    return p


def _fp8_ptrs(codes, scales, rows: int, K: int, name: str, dev: int):
    # the sizes of mmact_fp8_size; the codes' dtype is the format; _dev says what else is wrong
    code = FP8_DTYPE.get(codes.dtype) if isinstance(codes, torch.Tensor) else None
    if code is None:
        _dev(codes, name + " codes", _F8)
    pc, ps = _on(codes, name + " codes", codes.dtype, dev), _on(scales, name + " scales", torch.uint8, dev)
    if codes.numel() != rows * ((K + 15) // 16 * 16):
        raise ValueError(f"{name} codes must hold {rows} x {(K + 15) // 16 * 16} bytes")
    if scales.numel() != (rows + 127) // 128 * ((K + 511) // 512) * 512:
        raise ValueError(f"{name} scales must hold {(rows + 127) // 128} x {(K + 511) // 512} tiles of 512 bytes")
    return pc, ps, code


def mmact_quantize_fp8(x, codes, scales, block_rows: int = 1, transposed: bool = False, stream=None) -> None:
    """Quantise x [rows, K] (or, transposed, [K, rows]) to 8 bits with a scale for 128 values along K,
    or (block_rows 128) for 128 x 128; codes is a float8_e4m3fn or float8_e5m2 tensor and scales a uint8
    tensor of mmact_fp8_size(rows, K) bytes."""
    dev = _device(x, "x")
    px, dt, rows, K = _matrix_on(x, "x", dev)
    if transposed:
        rows, K = K, rows
    pc, ps, kind = _fp8_ptrs(codes, scales, rows, K, "x", dev)
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    s = (_lib or load()).mmact_quantize_fp8(px, pc, ps, rows, K, dt, kind, block_rows, 1 if transposed else 0,
                                            _stream_handle(stream))
    if s:
        _check(s, "mmact_quantize_fp8")


def mmact_dequantize_fp8(codes, scales, y, stream=None) -> None:
    """y [rows, K] = the values of an 8-bit matrix."""
    dev = _device(codes, "codes")
    py, dt, rows, K = _matrix_on(y, "y", dev)
    pc, ps, kind = _fp8_ptrs(codes, scales, rows, K, "y", dev)
    s = (_lib or load()).mmact_dequantize_fp8(pc, ps, py, rows, K, kind, dt, _stream_handle(stream))
    if s:
        _check(s, "mmact_dequantize_fp8")


def mmact_gemm_fp8(a_codes, a_scales, b_codes, b_scales, bias, C, K: int, act: str = "none", alpha: float = 0.0,
                   stream=None) -> None:
    """C = act(A @ B.T + bias) of 8-bit matrices A [M, K] and B [N, K]; C [M, N]."""
    dev = _device(a_codes, "a_codes")
    pc, dt, M, N = _matrix_on(C, "C", dev)
    pa, psa, ka = _fp8_ptrs(a_codes, a_scales, M, K, "A", dev)
    pb, psb, kb = _fp8_ptrs(b_codes, b_scales, N, K, "B", dev)
    s = (_lib or load()).mmact_gemm_fp8(pa, psa, pb, psb, _bias_on(bias, N, dev), pc, M, N, K, ka, kb, dt, ACT[act], alpha,
                                        _stream_handle(stream))
    if s:
        _check(s, "mmact_gemm_fp8")


def mmact_set_gemm_fp8_kernel(mode: int) -> None:
    """8-bit products: 0 kernel chosen per shape; 1 few rows or tiles; 2 CTA pairs."""
    _check(load().mmact_set_gemm_fp8_kernel(int(mode)), "mmact_set_gemm_fp8_kernel")


def mmact_linear_fp8_workspace_bytes(M: int, K: int) -> int:
    """Bytes of the workspace that mmact_linear_fp8 needs for x [M, K]."""
    out = ctypes.c_int64(0)
    _check(load().mmact_linear_fp8_workspace_bytes(int(M), int(K), ctypes.byref(out)), "mmact_linear_fp8_workspace_bytes")
    return out.value


def mmact_linear_fp8(x, w_codes, w_scales, bias, C, workspace, act: str = "none", alpha: float = 0.0,
                     stream=None) -> None:
    """C = act(q(x) @ W.T + bias): x [M, K] is quantised to E4M3 on the way in, W [N, K] is held in 8 bits."""
    dev = _device(x, "x")
    px, xd, M, K = _matrix_on(x, "x", dev)
    pc, cd, rows, N = _matrix_on(C, "C", dev)
    if rows != M:
        raise ValueError("x must be [M, K] and C [M, N]")
    pw, ps, kw = _fp8_ptrs(w_codes, w_scales, N, K, "W", dev)
    pws = _on(workspace, "workspace", torch.uint8, dev)
    if workspace.numel() < -(-M * ((K + 15) // 16 * 16) // 512) * 512 + (M + 127) // 128 * ((K + 511) // 512) * 512:
        raise ValueError("workspace must hold mmact_linear_fp8_workspace_bytes(M, K) bytes")
    s = (_lib or load()).mmact_linear_fp8(px, pw, ps, _bias_on(bias, N, dev), pc, M, N, K, xd, kw, cd, ACT[act], alpha, pws,
                                          _stream_handle(stream))
    if s:
        _check(s, "mmact_linear_fp8")


def mmact_linear_fp8_backward_workspace_bytes(M: int, N: int, K: int) -> int:
    """Bytes of the workspace that mmact_linear_fp8_backward needs for x [M, K] and dy [M, N]."""
    out = ctypes.c_int64(0)
    _check(load().mmact_linear_fp8_backward_workspace_bytes(int(M), int(N), int(K), ctypes.byref(out)),
           "mmact_linear_fp8_backward_workspace_bytes")
    return out.value


_F8_BACKWARD_WORKSPACE: dict = {}


def mmact_linear_fp8_backward(dy, x, wt_codes, wt_scales, dx, dw, db, workspace, grad_type=torch.float8_e5m2,
                              stream=None) -> None:
    """Gradients of x @ W.T + bias in 8 bits (see include/mmact.h): dy [M, N] and x [M, K] of one dtype, Wt
    [K, N] = W turned round in 8 bits; dx [M, K] of x's dtype, dw [N, K], db [N] float32, each may be None.
    dy is quantised to grad_type, x to E4M3."""
    dev = _device(dy, "dy")
    pdy, xd, M, N = _matrix_on(dy, "dy", dev)
    px, xd2, rows, K = _matrix_on(x, "x", dev)
    if rows != M or xd2 != xd:
        raise ValueError("dy must be [M, N] and x [M, K] of the same dtype")
    if grad_type not in FP8_DTYPE:
        raise TypeError(f"grad_type {grad_type} not in {_F8}")
    pdx = pdw = pdb = pw = ps = None
    kw, wd = FP8_DTYPE[torch.float8_e4m3fn], DTYPE[torch.float32]
    if dx is not None:
        pdx = _on(dx, "dx", x.dtype, dev)
        if dx.shape != x.shape:
            raise ValueError("dx must be [M, K]")
        pw, ps, kw = _fp8_ptrs(wt_codes, wt_scales, K, N, "Wt", dev)
    if dw is not None:
        pdw, wd, r, c = _matrix_on(dw, "dw", dev)
        if r != N or c != K:
            raise ValueError("dw must be [N, K]")
    if db is not None:
        pdb = _on(db, "db", torch.float32, dev)
        if db.dim() != 1 or db.shape[0] != N:
            raise ValueError("db must be [N]")
    pws = _on(workspace, "workspace", torch.uint8, dev)
    need = _F8_BACKWARD_WORKSPACE.get((M, N, K))
    if need is None:
        if len(_F8_BACKWARD_WORKSPACE) > 1024:
            _F8_BACKWARD_WORKSPACE.clear()
        need = _F8_BACKWARD_WORKSPACE[M, N, K] = mmact_linear_fp8_backward_workspace_bytes(M, N, K)
    if workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    s = (_lib or load()).mmact_linear_fp8_backward(pdy, px, pw, ps, pdx, pdw, pdb, M, N, K, xd, kw, FP8_DTYPE[grad_type], wd,
                                                   pws, _stream_handle(stream))
    if s:
        _check(s, "mmact_linear_fp8_backward")


def mmact_moe_workspace_bytes(T: int, H: int, I: int, E: int, top: int) -> int:
    """Bytes of the workspace that mmact_moe needs."""
    out = ctypes.c_int64(0)
    _check(load().mmact_moe_workspace_bytes(int(T), int(H), int(I), int(E), int(top), ctypes.byref(out)),
           "mmact_moe_workspace_bytes")
    return out.value


_MOE_WORKSPACE: dict = {}


def _f32_ptr(t, shape, name: str):
    if t is None:
        return None
    p = _dev(t, name, (torch.float32,))
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return p


def mmact_moe(x, router, w1, w2, y, experts, probs, workspace, act: str = "silu", alpha: float = 0.0,
              gated: bool = True, normalize: bool = True, router_bias=None, b1=None, b2=None, w1_scales=None,
              w2_scales=None, stream=None) -> None:
    """A whole mixture-of-experts layer for a few tokens (see include/mmact.h): x [T, H], router [E, H],
    y [T, H]; w1 [E, 2 I or I, H] and w2 [E, H, I] in x's dtype, or, with w1_scales and w2_scales, the
    codes of MXFP4 matrices [E * (2 I or I), H] and [E * H, I]; experts [T, top] int32 and probs
    [T, top] float32 are outputs."""
    L = load()
    io = (torch.float16, torch.bfloat16)
    px, pr, py = _dev(x, "x", io), _dev(router, "router", io), _dev(y, "y", io)
    pe, pp = _dev(experts, "experts", (torch.int32,)), _dev(probs, "probs", (torch.float32,))
    if x.dim() != 2 or router.dim() != 2 or router.shape[1] != x.shape[1] or y.shape != x.shape:
        raise ValueError("x must be [T, H], router [E, H] and y [T, H]")
    if router.dtype != x.dtype or y.dtype != x.dtype:
        raise ValueError("x, router and y must have the same dtype")
    T, H = x.shape
    E = router.shape[0]
    if experts.dim() != 2 or experts.shape[0] != T or probs.shape != experts.shape:
        raise ValueError("experts and probs must be [T, top]")
    top = experts.shape[1]
    halves = 2 if gated else 1
    mx = w1_scales is not None or w2_scales is not None
    if mx:
        if w1_scales is None or w2_scales is None:
            raise ValueError("w1_scales and w2_scales go together")
        row = (H + 31) // 32 * 16                   # bytes of one row of w1's codes
        if E == 0 or H == 0 or w1.numel() % (E * halves * row):
            raise ValueError("w1 must be the codes of an MXFP4 matrix [E * rows, H]")
        I = w1.numel() // (E * halves * row)
        p1, ps1 = _mxfp4_ptrs(w1, w1_scales, E * halves * I, H, "w1")
        p2, ps2 = _mxfp4_ptrs(w2, w2_scales, E * H, I, "w2")
        wd = MMACT_MXFP4
    else:
        p1, p2, ps1, ps2 = _dev(w1, "w1", (x.dtype,)), _dev(w2, "w2", (x.dtype,)), None, None
        if w1.dim() != 3 or w2.dim() != 3 or w1.shape[0] != E or w1.shape[2] != H or tuple(w2.shape[:2]) != (E, H):
            raise ValueError("w1 must be [E, rows, H] and w2 [E, H, I]")
        I = w2.shape[2]
        if w1.shape[1] != halves * I:
            raise ValueError("w1 must have 2 * I rows for each expert (gated), or I")
        wd = DTYPE[x.dtype]
    pws = _dev(workspace, "workspace", _BYTES)
    key = (T, H, I, E, top)
    need = _MOE_WORKSPACE.get(key)
    if need is None:
        if len(_MOE_WORKSPACE) > 1024:
            _MOE_WORKSPACE.clear()
        need = _MOE_WORKSPACE[key] = mmact_moe_workspace_bytes(*key)
    if workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    _check(L.mmact_moe(px, pr, _f32_ptr(router_bias, (E,), "router_bias"), p1, ps1,
                       _f32_ptr(b1, (E, halves * I), "b1"), p2, ps2, _f32_ptr(b2, (E, H), "b2"), py, pe, pp, T, H, I, E,
                       top, DTYPE[x.dtype], wd, ACT[act], float(alpha), 1 if gated else 0, 1 if normalize else 0, pws,
                       _stream_handle(stream)), "mmact_moe")


def mmact_moe_route_workspace_bytes(T: int, E: int) -> int:
    """Bytes of the workspace that mmact_moe_route needs."""
    out = ctypes.c_int64(0)
    _check(load().mmact_moe_route_workspace_bytes(int(T), int(E), ctypes.byref(out)), "mmact_moe_route_workspace_bytes")
    return out.value


_ROUTE_WORKSPACE: dict = {}


def _route_args(logits, mask, experts, counts, dev: int):
    pz, dt, T, E = _matrix_on(logits, "logits", dev)
    pe, pc = _on(experts, "experts", torch.int32, dev), _on(counts, "counts", torch.int32, dev)
    if experts.dim() != 2 or experts.shape[0] != T:
        raise ValueError("experts must be [T, top]")
    if counts.numel() != E + 1:
        raise ValueError("counts must be [E + 1]")
    pm = None
    if mask is not None:
        pm = _on(mask, "mask", torch.bool if mask.dtype is torch.bool else torch.uint8, dev)
        if mask.dim() != 1 or mask.shape[0] != T:
            raise ValueError("mask must be [T]")
    return pz, pm, pe, pc, T, E, experts.shape[1], dt


def _one_on(t, name: str, dev: int) -> int:
    p = _on(t, name, torch.float32, dev)
    if t.numel() != 1:
        raise ValueError(f"{name} must have one element")
    return p


def mmact_moe_route(logits, experts, probs, counts, loss, workspace, coef: float = 1.0, normalize: bool = True, mask=None,
                    stream=None) -> None:
    """A router in training (see include/mmact.h): from logits [T, E] the outputs experts [T, top] int32, probs
    [T, top] float32, counts [E + 1] int32 and loss [1] float32; mask [T] uint8 or bool leaves out tokens."""
    dev = _device(logits, "logits")
    pz, pm, pe, pc, T, E, top, dt = _route_args(logits, mask, experts, counts, dev)
    pp, pl = _on(probs, "probs", torch.float32, dev), _one_on(loss, "loss", dev)
    if probs.shape != experts.shape:
        raise ValueError("experts and probs must be [T, top]")
    pws = _on(workspace, "workspace", torch.uint8, dev)
    need = _ROUTE_WORKSPACE.get((T, E))
    if need is None:
        if len(_ROUTE_WORKSPACE) > 1024:
            _ROUTE_WORKSPACE.clear()
        need = _ROUTE_WORKSPACE[T, E] = mmact_moe_route_workspace_bytes(T, E)
    if workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    s = (_lib or load()).mmact_moe_route(pz, pm, pe, pp, pc, pl, T, E, top, dt, 1 if normalize else 0, coef, pws,
                                         _stream_handle(stream))
    if s:
        _check(s, "mmact_moe_route")


def mmact_moe_route_backward(logits, experts, counts, dprobs, dloss, dlogits, coef: float = 1.0, normalize: bool = True,
                             mask=None, stream=None) -> None:
    """The gradient dlogits [T, E] of mmact_moe_route's logits from dprobs [T, top] and dloss [1] (float32, either
    may be None); logits, experts, counts, coef, normalize and mask are the forward pass's."""
    dev = _device(logits, "logits")
    pz, pm, pe, pc, T, E, top, dt = _route_args(logits, mask, experts, counts, dev)
    pd = _on(dlogits, "dlogits", logits.dtype, dev)
    if dlogits.shape != logits.shape:
        raise ValueError("dlogits must be [T, E]")
    pg = pl = None
    if dprobs is not None:
        pg = _on(dprobs, "dprobs", torch.float32, dev)
        if dprobs.shape != experts.shape:
            raise ValueError("dprobs must be [T, top]")
    if dloss is not None:
        pl = _one_on(dloss, "dloss", dev)
    s = (_lib or load()).mmact_moe_route_backward(pz, pm, pe, pc, pg, pl, pd, T, E, top, dt, 1 if normalize else 0, coef,
                                                  _stream_handle(stream))
    if s:
        _check(s, "mmact_moe_route_backward")


def mmact_get_last_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word's verdict."""
    return int(load().mmact_get_last_error(_stream_handle(stream)))


def mmact_set_wait_timeout_ns(ns: int) -> None:
    load().mmact_set_wait_timeout_ns(int(ns))


def mmact_selftest_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check(load().mmact_selftest_wait_timeout(int(timeout_ns), _stream_handle(stream)),
           "mmact_selftest_wait_timeout")


def mmact_set_gemm_tile_n(tile_n: int) -> None:
    _check(load().mmact_set_gemm_tile_n(int(tile_n)), "mmact_set_gemm_tile_n")


def mmact_set_gemm_split_k(split_k: int) -> None:
    """0: split-K chosen per shape; 1: never; 2 or 4: whenever legal."""
    _check(load().mmact_set_gemm_split_k(int(split_k)), "mmact_set_gemm_split_k")


def mmact_set_gemm_pair(mode: int) -> None:
    """CTA-pair GEMM kernel: 0 chosen per shape; 1 never; 2 always (when split-K is not taken)."""
    _check(load().mmact_set_gemm_pair(int(mode)), "mmact_set_gemm_pair")


def mmact_set_conv_tmem(mode: int) -> None:
    """NCHW conv with the im2col operand in tensor memory: 0 where it applies (default); 1 never."""
    _check(load().mmact_set_conv_tmem(int(mode)), "mmact_set_conv_tmem")


def mmact_set_gemm_l2_policy(mode: int) -> None:
    """CTA-pair GEMM: 1 A evict-last and C evict-first in L2 (default); 0 no cache hints."""
    _check(load().mmact_set_gemm_l2_policy(int(mode)), "mmact_set_gemm_l2_policy")


def mmact_tensor_map_cache_stats() -> tuple[int, int]:
    """(hits, encodes) of the library's host-side tensor-map cache, process-wide."""
    h, e = ctypes.c_uint64(0), ctypes.c_uint64(0)
    _check(load().mmact_tensor_map_cache_stats(ctypes.byref(h), ctypes.byref(e)), "mmact_tensor_map_cache_stats")
    return int(h.value), int(e.value)


GEMM_KERNELS = {0: "none", 1: "persistent", 2: "pair", 3: "split_k"}


def mmact_gemm_kernel_choice(M: int, N: int, K: int, residual: bool = False) -> str:
    """The kernel a GEMM of this shape would run: "none", "persistent", "pair" or "split_k"."""
    out = ctypes.c_int(-1)
    _check(load().mmact_gemm_kernel_choice(int(M), int(N), int(K), 1 if residual else 0,
                                           ctypes.byref(out)), "mmact_gemm_kernel_choice")
    return GEMM_KERNELS[out.value]


def mmact_gemm_split_k_choice(M: int, N: int, K: int) -> int:
    """Split-K factor (0, 2 or 4) a GEMM of this shape would use on the current device."""
    out = ctypes.c_int(-1)
    _check(load().mmact_gemm_split_k_choice(int(M), int(N), int(K), ctypes.byref(out)),
           "mmact_gemm_split_k_choice")
    return out.value


def mmact_status_string(status: int) -> str:
    return status_string(status)


def mmact_version() -> int:
    return int(load().mmact_version())
