"""OCP-MX block quantization (MXFP4 / MXFP8) on GB300: Python binding of libmxq.

Every function here has the name of the C entry point it calls (include/mxq.h) and does
argument marshalling only: it checks tensor device/dtype/shape, allocates outputs with torch
when the caller passes none, and hands raw device pointers and the current CUDA stream to the
library. All computation runs in the library's sm_103a kernels. If libmxq.so is missing the
calls raise; there is no fallback. No call records anything for autograd: results are cut from the
graph of their inputs, gradients have calls of their own (examples/expert_layer.py joins them).
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

E2M1 = MXFP4 = 1
E4M3 = MXFP8 = 2
LINEAR = 0
SWIZZLED = 1
RNE = 0    # abs-max block scale
QUEST = 1  # Quest-like block scale (clip point alpha * RMS), MXFP4 only, not grouped
GROUP = 32
ROT_DENSE = 0     # any H: tensor-core product
ROT_HADAMARD = 1  # H = H[0][0] * Sylvester (stated by the caller, checked on the device)
ROT_AUTO = 2      # the same statement; the library takes the kernel measured faster for the call

SOFTMAX, SIGMOID = 0, 1          # scores of mx_route
B128_BLOCKS, B128_ROWS = 0, 1    # forms of B's scales in mx_gemm_b128
BLOCK128 = 128

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxq.so")
_lib = None

EXPORTS = (
    "mx_status_string", "mx_scales_shape", "mx_grouped_scales_shape", "mx_quantize", "mx_qdq",
    "mx_rotate_quantize", "mx_quantize_grouped", "mx_dequantize", "mx_nvfp4_scales_shape",
    "mx_quantize_nvfp4", "mx_qdq_nvfp4", "mx_dequantize_nvfp4", "mx_nvfp4_grouped_scales_shape",
    "mx_quantize_nvfp4_grouped", "mx_rotate_debug", "mx_device_errors",
    "mx_selftest_bounded_wait", "mx_selftest_rotate_give_up", "mx_gemm",
    "mx_selftest_gemm_give_up", "mx_route", "mx_route_backward", "mx_route_plan_workspace",
    "mx_route_plan", "mx_b128_padded_rows", "mx_quantize_b128_rows", "mx_quantize_b128_cols",
    "mx_quantize_b128_blocks", "mx_gemm_b128", "mx_gemm_b128_grouped",
    "mx_gemm_b128_grouped_wgrad", "mx_combine", "mx_combine_backward",
    "mx_combine_backward_whole",
    "mx_selftest_gemm_b128_give_up", "mx_selftest_gemm_b128_grouped_give_up",
)


class MXError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libmxq (ctypes handle with argument types set)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m mx_microscaling_quantize_gb300._build` "
            "(or __graft_entry__.build()) first")
    L = ctypes.CDLL(LIB_PATH)
    i32, i64, p = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
    pi64 = ctypes.POINTER(ctypes.c_int64)
    sigs = {
        "mx_status_string": (ctypes.c_char_p, [i32]),
        "mx_scales_shape": (i32, [i64, i64, i32, i32, pi64, pi64]),
        "mx_grouped_scales_shape": (i32, [i64, i32, i64, i32, i32, pi64, pi64]),
        "mx_quantize": (i32, [p, i64, i64, i32, i32, i32, i32, p, p, p]),
        "mx_qdq": (i32, [p, i64, i64, i32, i32, i32, p, i32, i32, p, p]),
        "mx_rotate_quantize": (i32, [p, i64, i64, p, i32, i32, i32, i32, i32, i32, p, p, p]),
        "mx_quantize_grouped": (i32, [p, p, i32, i64, i64, i32, i32, i32, i32, p, p, p]),
        "mx_dequantize": (i32, [p, p, i64, i64, i32, i32, i32, p, p]),
        "mx_nvfp4_scales_shape": (i32, [i64, i64, i32, pi64, pi64]),
        "mx_quantize_nvfp4": (i32, [p, i64, i64, p, i32, i32, p, i32, p, p, p]),
        "mx_qdq_nvfp4": (i32, [p, i64, i64, p, i32, i32, p, p, p]),
        "mx_dequantize_nvfp4": (i32, [p, p, i64, i64, p, i32, p, p]),
        "mx_nvfp4_grouped_scales_shape": (i32, [i64, i32, i64, i32, pi64, pi64]),
        "mx_quantize_nvfp4_grouped": (i32, [p, p, i32, i64, i64, p, i32, p, p, p]),
        "mx_rotate_debug": (i32, [p, i64, i64, p, i32, i32, p, p]),
        "mx_device_errors": (i32, [ctypes.POINTER(ctypes.c_int)]),
        "mx_selftest_bounded_wait": (i32, [i64, p]),
        "mx_selftest_rotate_give_up": (i32, [p, i64, i64, p, i32, p, p, i64, p]),
        "mx_gemm": (i32, [p, p, p, p, i64, i64, i64, i32, i32, i32, ctypes.c_float, p, p]),
        "mx_selftest_gemm_give_up": (i32, [p, p, p, p, i64, i64, i64, i32, i32, p, i64, p]),
        "mx_route": (i32, [p, i32, p, i64, i32, i32, i32, i32, i32, i32, ctypes.c_float, p, p, p]),
        "mx_route_backward": (i32, [p, p, i32, p, i64, i32, i32, i32, i32, ctypes.c_float, p, p]),
        "mx_route_plan_workspace": (i32, [i64, i32, i32, pi64]),
        "mx_route_plan": (i32, [p, i64, i32, i32, p, p, p, p, p]),
        "mx_b128_padded_rows": (i32, [i64, i32, pi64]),
        "mx_quantize_b128_rows": (i32, [p, i64, i64, p, i64, p, p, p]),
        "mx_quantize_b128_cols": (i32, [p, i64, i64, p, i64, p, i32, p, p, p]),
        "mx_quantize_b128_blocks": (i32, [p, i64, i64, i64, p, p, p, p, p]),
        "mx_gemm_b128": (i32, [p, p, p, p, i64, i64, i64, i32, i32, p, p]),
        "mx_gemm_b128_grouped": (i32, [p, p, p, p, p, i32, i64, i64, i64, i32, p, p]),
        "mx_gemm_b128_grouped_wgrad": (i32, [p, p, p, p, p, i32, i64, i64, i64, i32, p, p]),
        "mx_combine": (i32, [p, p, p, i64, i32, i64, i64, p, p]),
        "mx_combine_backward": (i32, [p, p, p, p, i64, i32, i64, i64, p, p, p]),
        "mx_combine_backward_whole": (i32, [p, p, p, p, i64, i32, i64, i64, p, p, p, p]),
        "mx_selftest_gemm_b128_give_up": (i32, [p, p, p, p, i64, i64, i64, i32, p, i64, p]),
        "mx_selftest_gemm_b128_grouped_give_up": (i32, [p, p, p, p, p, i32, i64, i64, i64, p, i64, p]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def mx_status_string(status: int) -> str:
    return lib().mx_status_string(status).decode()


def _check(status: int) -> None:
    if status != 0:
        raise MXError(status, mx_status_string(status))


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream, t: torch.Tensor) -> int:
    """The cudaStream_t to launch on: `stream` (a torch.cuda.Stream or a raw handle), or when
    None the current stream of t's device (read without building a Stream object, which costs
    microseconds per call)."""
    if stream is None:
        dev = t.get_device()
        if _raw_stream is not None:
            return _raw_stream(dev)
        return torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _as_stream(stream, device) -> torch.cuda.Stream:
    """`stream` (a torch.cuda.Stream or a raw handle) as a stream that torch can allocate under."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    # the handle 1 names the default stream, as 0 does; torch knows it by 0 only
    return torch.cuda.ExternalStream(0 if stream == 1 else stream, device)


def _empty(shape, dtype, like: torch.Tensor, stream, scratch: bool = False) -> torch.Tensor:
    """Device memory for a call on `stream`, taken from that stream's pool: a block of another stream's
    may still be in use by what is queued there. The current stream, where a caller goes on with an
    output, is recorded: the block is not handed on before what is queued there by the time it is freed.
    A call's own scratch memory is used on `stream` alone."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(_as_stream(stream, like.device)):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    if not scratch:
        t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _input(x: torch.Tensor, name: str = "x") -> tuple[int, int]:
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.bfloat16):
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D [M, K] tensor")
    return x.shape[0], x.shape[1]


def _rotation(H: torch.Tensor) -> int:
    if not (isinstance(H, torch.Tensor) and H.is_cuda and H.dtype == torch.bfloat16):
        raise TypeError("H must be a CUDA bfloat16 tensor")
    if H.dim() != 2 or H.shape[0] != H.shape[1] or not H.is_contiguous():
        raise ValueError("H must be a contiguous square [g, g] tensor")
    return H.shape[0]


def code_bytes_per_row(fmt: int, K: int) -> int:
    return K if fmt == E4M3 else K // 2


def _codes_out(codes, x, M, K, fmt, stream):
    if codes is None:
        return _empty((M, code_bytes_per_row(fmt, K)), torch.uint8, x, stream)
    if codes.numel() * codes.element_size() != M * code_bytes_per_row(fmt, K):
        raise ValueError("codes has the wrong size")
    return codes


def _scales_out(scales, x, shape, stream):
    rows, cols = shape
    if scales is None:
        return _empty((rows, cols), torch.uint8, x, stream)
    if scales.numel() * scales.element_size() != rows * cols:
        raise ValueError("scales has the wrong size")
    return scales


@functools.lru_cache(maxsize=4096)
def mx_scales_shape(M: int, K: int, layout: int = LINEAR, group: int = GROUP) -> tuple[int, int]:
    r, c = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().mx_scales_shape(M, K, group, layout, ctypes.byref(r), ctypes.byref(c)))
    return r.value, c.value


@functools.lru_cache(maxsize=4096)
def mx_grouped_scales_shape(M_total: int, E: int, K: int, layout: int = SWIZZLED,
                            group: int = GROUP) -> tuple[int, int]:
    r, c = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().mx_grouped_scales_shape(M_total, E, K, group, layout, ctypes.byref(r),
                                         ctypes.byref(c)))
    return r.value, c.value


def mx_quantize(x, fmt, layout=LINEAR, *, codes=None, scales=None, group=GROUP, rounding=RNE,
                stream=None):
    """Block quantize bf16 [M, K] -> (codes uint8, E8M0 scales uint8)."""
    M, K = _input(x)
    codes = _codes_out(codes, x, M, K, fmt, stream)
    scales = _scales_out(scales, x, mx_scales_shape(M, K, layout, group), stream)
    _check(lib().mx_quantize(_ptr(x), M, K, fmt, group, layout, rounding, _ptr(codes),
                             _ptr(scales), _stream_ptr(stream, x)))
    return codes, scales


def mx_qdq(x, fmt, H=None, *, y=None, group=GROUP, rounding=RNE, rot_kind=ROT_DENSE,
           stream=None):
    """Quantize-dequantize bf16 [M, K] -> bf16 [M, K]; with H, rotate each g-chunk first
    (rot_kind: ROT_DENSE, ROT_HADAMARD or ROT_AUTO)."""
    M, K = _input(x)
    g = _rotation(H) if H is not None else 0
    if y is None:
        y = _empty(x.shape, x.dtype, x, stream)
    _check(lib().mx_qdq(_ptr(x), M, K, fmt, group, rounding, _ptr(H), g, rot_kind, _ptr(y),
                        _stream_ptr(stream, x)))
    return y


def mx_rotate_quantize(x, H, fmt, layout=SWIZZLED, *, codes=None, scales=None, group=GROUP,
                       rounding=RNE, rot_kind=ROT_DENSE, stream=None):
    """Rotate each g-chunk by H, then block quantize -> (codes, scales)."""
    M, K = _input(x)
    g = _rotation(H)
    codes = _codes_out(codes, x, M, K, fmt, stream)
    scales = _scales_out(scales, x, mx_scales_shape(M, K, layout, group), stream)
    _check(lib().mx_rotate_quantize(_ptr(x), M, K, _ptr(H), g, rot_kind, fmt, group, layout,
                                    rounding, _ptr(codes), _ptr(scales), _stream_ptr(stream, x)))
    return codes, scales


def mx_quantize_grouped(x, row_offsets, fmt, layout=SWIZZLED, *, codes=None, scales=None,
                        group=GROUP, rounding=RNE, stream=None):
    """Per-expert block quantize; row_offsets: CUDA int64 [E + 1]."""
    M, K = _input(x)
    if not (row_offsets.is_cuda and row_offsets.dtype == torch.int64 and row_offsets.dim() == 1
            and row_offsets.is_contiguous()):
        raise TypeError("row_offsets must be a contiguous CUDA int64 [E + 1] tensor")
    E = row_offsets.numel() - 1
    codes = _codes_out(codes, x, M, K, fmt, stream)
    scales = _scales_out(scales, x, mx_grouped_scales_shape(M, E, K, layout, group), stream)
    _check(lib().mx_quantize_grouped(_ptr(x), _ptr(row_offsets), E, M, K, fmt, group, layout,
                                     rounding, _ptr(codes), _ptr(scales), _stream_ptr(stream, x)))
    return codes, scales


def mx_dequantize(codes, scales, K, fmt, layout=LINEAR, *, y=None, group=GROUP, stream=None):
    """Stored codes (uint8 [M, K or K/2]) and E8M0 scales -> bf16 [M, K]."""
    if not (isinstance(codes, torch.Tensor) and codes.is_cuda and codes.dim() == 2
            and codes.is_contiguous() and codes.element_size() == 1):
        raise TypeError("codes must be a contiguous CUDA 2-D tensor of bytes")
    if not (isinstance(scales, torch.Tensor) and scales.is_cuda and scales.is_contiguous()
            and scales.element_size() == 1):
        raise TypeError("scales must be a contiguous CUDA tensor of bytes")
    M = codes.shape[0]
    if codes.shape[1] != code_bytes_per_row(fmt, K):
        raise ValueError("codes has the wrong row length for K and fmt")
    rows, cols = mx_scales_shape(M, K, layout, group)
    if scales.numel() != rows * cols:
        raise ValueError("scales has the wrong size")
    if y is None:
        y = _empty((M, K), torch.bfloat16, codes, stream)
    elif not (y.is_cuda and y.dtype == torch.bfloat16 and y.numel() == M * K
              and y.is_contiguous()):
        raise ValueError("y must be a contiguous CUDA bfloat16 tensor of M * K elements")
    _check(lib().mx_dequantize(_ptr(codes), _ptr(scales), M, K, fmt, group, layout, _ptr(y),
                               _stream_ptr(stream, codes)))
    return y


@functools.lru_cache(maxsize=4096)
def mx_nvfp4_scales_shape(M: int, K: int, layout: int = SWIZZLED) -> tuple[int, int]:
    r, c = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().mx_nvfp4_scales_shape(M, K, layout, ctypes.byref(r), ctypes.byref(c)))
    return r.value, c.value


def _global_scale(gs) -> None:
    if not (isinstance(gs, torch.Tensor) and gs.is_cuda and gs.dtype == torch.float32
            and gs.numel() == 1):
        raise TypeError("global_scale must be a CUDA float32 tensor of one element")


def mx_quantize_nvfp4(x, global_scale, layout=SWIZZLED, H=None, *, codes=None, scales=None,
                      rot_kind=ROT_DENSE, stream=None):
    """NVFP4 quantize (optionally rotating each g-chunk by H first) -> (codes, E4M3 scales)."""
    M, K = _input(x)
    _global_scale(global_scale)
    g = _rotation(H) if H is not None else 0
    codes = _codes_out(codes, x, M, K, E2M1, stream)
    scales = _scales_out(scales, x, mx_nvfp4_scales_shape(M, K, layout), stream)
    _check(lib().mx_quantize_nvfp4(_ptr(x), M, K, _ptr(H), g, rot_kind, _ptr(global_scale),
                                   layout, _ptr(codes), _ptr(scales), _stream_ptr(stream, x)))
    return codes, scales


def mx_qdq_nvfp4(x, global_scale, H=None, *, y=None, rot_kind=ROT_DENSE, stream=None):
    """NVFP4 quantize-dequantize bf16 [M, K] -> bf16 [M, K] (optionally rotated)."""
    M, K = _input(x)
    _global_scale(global_scale)
    g = _rotation(H) if H is not None else 0
    if y is None:
        y = _empty(x.shape, x.dtype, x, stream)
    _check(lib().mx_qdq_nvfp4(_ptr(x), M, K, _ptr(H), g, rot_kind, _ptr(global_scale), _ptr(y),
                              _stream_ptr(stream, x)))
    return y


@functools.lru_cache(maxsize=4096)
def mx_nvfp4_grouped_scales_shape(M_total: int, E: int, K: int,
                                  layout: int = SWIZZLED) -> tuple[int, int]:
    r, c = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().mx_nvfp4_grouped_scales_shape(M_total, E, K, layout, ctypes.byref(r),
                                               ctypes.byref(c)))
    return r.value, c.value


def mx_quantize_nvfp4_grouped(x, row_offsets, global_scales, layout=SWIZZLED, *, codes=None,
                              scales=None, stream=None):
    """Per-expert NVFP4 quantize; row_offsets: CUDA int64 [E + 1]; global_scales: CUDA fp32 [E]."""
    M, K = _input(x)
    if not (row_offsets.is_cuda and row_offsets.dtype == torch.int64 and row_offsets.dim() == 1
            and row_offsets.is_contiguous()):
        raise TypeError("row_offsets must be a contiguous CUDA int64 [E + 1] tensor")
    E = row_offsets.numel() - 1
    if not (isinstance(global_scales, torch.Tensor) and global_scales.is_cuda
            and global_scales.dtype == torch.float32 and global_scales.numel() == E
            and global_scales.is_contiguous()):
        raise TypeError("global_scales must be a contiguous CUDA float32 tensor of E elements")
    codes = _codes_out(codes, x, M, K, E2M1, stream)
    scales = _scales_out(scales, x, mx_nvfp4_grouped_scales_shape(M, E, K, layout), stream)
    _check(lib().mx_quantize_nvfp4_grouped(_ptr(x), _ptr(row_offsets), E, M, K,
                                           _ptr(global_scales), layout, _ptr(codes),
                                           _ptr(scales), _stream_ptr(stream, x)))
    return codes, scales


def mx_dequantize_nvfp4(codes, scales, K, global_scale, layout=SWIZZLED, *, y=None,
                        stream=None):
    """Stored NVFP4 codes (uint8 [M, K/2]) and E4M3 scales -> bf16 [M, K]."""
    if not (isinstance(codes, torch.Tensor) and codes.is_cuda and codes.dim() == 2
            and codes.is_contiguous() and codes.element_size() == 1):
        raise TypeError("codes must be a contiguous CUDA 2-D tensor of bytes")
    if not (isinstance(scales, torch.Tensor) and scales.is_cuda and scales.is_contiguous()
            and scales.element_size() == 1):
        raise TypeError("scales must be a contiguous CUDA tensor of bytes")
    _global_scale(global_scale)
    M = codes.shape[0]
    if codes.shape[1] != K // 2:
        raise ValueError("codes has the wrong row length for K")
    rows, cols = mx_nvfp4_scales_shape(M, K, layout)
    if scales.numel() != rows * cols:
        raise ValueError("scales has the wrong size")
    if y is None:
        y = _empty((M, K), torch.bfloat16, codes, stream)
    elif not (y.is_cuda and y.dtype == torch.bfloat16 and y.numel() == M * K
              and y.is_contiguous()):
        raise ValueError("y must be a contiguous CUDA bfloat16 tensor of M * K elements")
    _check(lib().mx_dequantize_nvfp4(_ptr(codes), _ptr(scales), M, K, _ptr(global_scale), layout,
                                     _ptr(y), _stream_ptr(stream, codes)))
    return y


def mx_rotate_debug(x, H, *, y=None, rot_kind=ROT_DENSE, stream=None):
    """The fp32 rotated values the rotated kernels quantize (diagnostics)."""
    M, K = _input(x)
    g = _rotation(H)
    if y is None:
        y = _empty((M, K), torch.float32, x, stream)
    _check(lib().mx_rotate_debug(_ptr(x), M, K, _ptr(H), g, rot_kind, _ptr(y),
                                 _stream_ptr(stream, x)))
    return y


def mx_device_errors() -> int:
    """Synchronize and return (then clear) the device error word."""
    v = ctypes.c_int()
    _check(lib().mx_device_errors(ctypes.byref(v)))
    return v.value


def mx_selftest_bounded_wait(limit_ns: int = 1_000_000, *, stream=None, device: int = 0) -> None:
    """Run one bounded wait that nothing completes (it gives up after limit_ns and sets the
    device error word; read it with mx_device_errors())."""
    st = stream
    if st is None:
        st = _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream
    elif isinstance(st, torch.cuda.Stream):
        st = st.cuda_stream
    _check(lib().mx_selftest_bounded_wait(limit_ns, st))


def mx_selftest_rotate_give_up(x, H, limit_ns: int, *, stream=None):
    """The tensor-core rotate + MXFP4 quantize (swizzled scales) with every wait of the kernel
    limited to limit_ns: waits run out while the pipeline is busy, the kernel stops issuing
    work, drains what is in flight and returns; the device error word reports it (read it with
    mx_device_errors()). Returns the (unspecified) codes and scales buffers."""
    M, K = _input(x)
    g = _rotation(H)
    codes = _codes_out(None, x, M, K, E2M1, stream)
    scales = _scales_out(None, x, mx_scales_shape(M, K, SWIZZLED), stream)
    _check(lib().mx_selftest_rotate_give_up(_ptr(x), M, K, _ptr(H), g, _ptr(codes), _ptr(scales),
                                            limit_ns, _stream_ptr(stream, x)))
    return codes, scales


def _gemm_operands(a_codes, a_scales, b_codes, b_scales, K, fmt, c, stream):
    for t in (a_codes, a_scales, b_codes, b_scales):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.uint8
                and t.is_contiguous()):
            raise TypeError("codes and scales must be contiguous CUDA uint8 tensors")
    M, N = a_codes.shape[0], b_codes.shape[0]
    if a_codes.numel() != M * code_bytes_per_row(fmt, K) or \
            b_codes.numel() != N * code_bytes_per_row(fmt, K):
        raise ValueError("codes do not match K and the format")
    if c is None:
        c = _empty((M, N), torch.bfloat16, a_codes, stream)
    return M, N, c


def mx_selftest_gemm_give_up(a_codes, a_scales, b_codes, b_scales, K: int, fmt, layout, limit_ns: int,
                             *, stream=None):
    """mx_gemm with every pipeline wait of the kernel limited to limit_ns: the kernel stops
    issuing work, drains what is in flight and returns; the device error word reports it.
    Returns the (unspecified) C buffer."""
    M, N, c = _gemm_operands(a_codes, a_scales, b_codes, b_scales, K, fmt, None, stream)
    _check(lib().mx_selftest_gemm_give_up(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes),
                                          _ptr(b_scales), M, N, K, fmt, layout, _ptr(c), limit_ns,
                                          _stream_ptr(stream, a_codes)))
    return c


def mx_gemm(a_codes, a_scales, b_codes, b_scales, K: int, fmt, layout=SWIZZLED, alpha: float = 1.0,
            *, c=None, group=GROUP, stream=None):
    """C[M, N] = alpha * dequant(A) @ dequant(B)^T (bf16) from MX codes and E8M0 scales as
    mx_quantize returns them (A: [M, K/2 or K] codes, B: [N, ...])."""
    M, N, c = _gemm_operands(a_codes, a_scales, b_codes, b_scales, K, fmt, c, stream)
    _check(lib().mx_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), M, N, K,
                         fmt, group, layout, alpha, _ptr(c), _stream_ptr(stream, a_codes)))
    return c


# ---------------------------------------------------------------------------------------------
# expert layers: routing, operands with a scale per block of 128, their products, combination
# ---------------------------------------------------------------------------------------------
_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def _tensor(t, name, dtype, *, dim=None, like=None) -> torch.Tensor:
    """A contiguous CUDA tensor of one of the dtypes (and dimensions), on like's device."""
    # The usual case first: the small calls take longer in Python than on the device.
    if type(t) is torch.Tensor and t.is_cuda and t.is_contiguous() and \
            (t.dtype is dtype or (dtype is _TYPES and t.dtype in dtype)) and \
            (dim is None or t.ndim == dim) and (like is None or t.get_device() == like.get_device()):
        return t
    dtypes = dtype if isinstance(dtype, (tuple, dict)) else (dtype,)
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes):
        raise TypeError(f"{name} must be a CUDA tensor of {' or '.join(map(str, dtypes))}")
    if not t.is_contiguous() or (dim is not None and t.dim() not in
                                 (dim if isinstance(dim, tuple) else (dim,))):
        raise ValueError(f"{name} must be contiguous" +
                         ("" if dim is None else f" with {dim} dimensions"))
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}")
    return t


def _output(t, name, shape, dtype, like, stream) -> torch.Tensor:
    """t checked against shape, or a new tensor of it on like's device."""
    if t is None:
        return _empty(shape, dtype, like, stream)
    _tensor(t, name, dtype, like=like)
    n = 1
    for d in shape:
        n *= d
    if t.numel() != n:
        raise ValueError(f"{name} has the wrong size")
    return t


def mx_route(logits, k: int, score=SOFTMAX, bias=None, *, groups: int = 1, top_groups: int = 1,
             renormalize: bool = True, scale: float = 1.0, experts=None, weights=None, stream=None):
    """Choose k experts per token from logits [T, E] (bfloat16 or float32) -> (experts int32
    [T, k], weights float32 [T, k]); experts of logit -inf are never chosen (-1, weight 0)."""
    _tensor(logits, "logits", _TYPES, dim=2)
    T, E = logits.shape
    if bias is not None and _tensor(bias, "bias", torch.float32, like=logits).numel() != E:
        raise ValueError("bias must have one value per expert")
    experts = _output(experts, "experts", (T, k), torch.int32, logits, stream)
    weights = _output(weights, "weights", (T, k), torch.float32, logits, stream)
    _check(lib().mx_route(_ptr(logits), _TYPES[logits.dtype], _ptr(bias), T, E, k, score, groups,
                          top_groups, int(renormalize), scale, _ptr(experts), _ptr(weights),
                          _stream_ptr(stream, logits)))
    return experts, weights


def mx_route_backward(grad_weights, logits, experts, score=SOFTMAX, *, renormalize: bool = True,
                      scale: float = 1.0, grad_logits=None, stream=None):
    """Gradient of the logits [T, E] from that of mx_route's weights [T, k]."""
    _tensor(logits, "logits", _TYPES, dim=2)
    _tensor(experts, "experts", torch.int32, dim=2, like=logits)
    _tensor(grad_weights, "grad_weights", torch.float32, dim=2, like=logits)
    T, E = logits.shape
    k = experts.shape[1]
    if experts.shape[0] != T or grad_weights.shape != experts.shape:
        raise ValueError("experts and grad_weights must be [T, k]")
    grad_logits = _output(grad_logits, "grad_logits", (T, E), logits.dtype, logits, stream)
    _check(lib().mx_route_backward(_ptr(grad_weights), _ptr(logits), _TYPES[logits.dtype],
                                   _ptr(experts), T, E, k, score, int(renormalize), scale,
                                   _ptr(grad_logits), _stream_ptr(stream, logits)))
    return grad_logits


@functools.lru_cache(maxsize=4096)
def mx_route_plan_workspace(T: int, k: int, E: int) -> int:
    """Bytes of device memory mx_route_plan works in."""
    n = ctypes.c_int64()
    _check(lib().mx_route_plan_workspace(T, k, E, ctypes.byref(n)))
    return n.value


def mx_route_plan(experts, E: int, *, row_offsets=None, tokens=None, slots=None, workspace=None,
                  stream=None):
    """Order the choices [T, k] by expert -> (row_offsets int64 [E + 1], tokens int32 [T * k],
    slots int32 [T, k])."""
    _tensor(experts, "experts", torch.int32, dim=2)
    T, k = experts.shape
    need = mx_route_plan_workspace(T, k, E)
    row_offsets = _output(row_offsets, "row_offsets", (E + 1,), torch.int64, experts, stream)
    tokens = _output(tokens, "tokens", (T * k,), torch.int32, experts, stream)
    slots = _output(slots, "slots", (T, k), torch.int32, experts, stream)
    if workspace is None:
        if need:
            workspace = _empty((need,), torch.uint8, experts, stream, scratch=True)
    elif workspace.device != experts.device or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must have {need} bytes on {experts.device}")
    _check(lib().mx_route_plan(_ptr(experts), T, k, E, _ptr(row_offsets), _ptr(tokens), _ptr(slots),
                               _ptr(workspace), _stream_ptr(stream, experts)))
    return row_offsets, tokens, slots


@functools.lru_cache(maxsize=4096)
def mx_b128_padded_rows(R: int, E: int = 1) -> int:
    """Columns of a mx_quantize_b128_cols operand of R rows of E experts."""
    n = ctypes.c_int64()
    _check(lib().mx_b128_padded_rows(R, E, ctypes.byref(n)))
    return n.value


def _row_index(index, x, M):
    if index is None:
        return M
    return _tensor(index, "index", torch.int32, dim=1, like=x).numel()


def _offsets(row_offsets, like) -> int:
    E = _tensor(row_offsets, "row_offsets", torch.int64, dim=1, like=like).numel() - 1
    if E < 1:
        raise ValueError("row_offsets must be [E + 1]")
    return E


def mx_quantize_b128_rows(x, index=None, *, codes=None, scales=None, stream=None):
    """bf16 [M, K] (rows `index` of it, int32 [R]) -> (E4M3 codes uint8 [R, K], scales float32
    [ceil(K / 128), R]), one scale per 128 elements of a row."""
    M, K = _input(x)
    R = _row_index(index, x, M)
    codes = _output(codes, "codes", (R, K), torch.uint8, x, stream)
    scales = _output(scales, "scales", (-(-K // BLOCK128), R), torch.float32, x, stream)
    _check(lib().mx_quantize_b128_rows(_ptr(x), M, K, _ptr(index), R, _ptr(codes), _ptr(scales),
                                       _stream_ptr(stream, x)))
    return codes, scales


def mx_quantize_b128_cols(x, index=None, row_offsets=None, *, codes=None, scales=None, stream=None):
    """bf16 [M, K] (rows `index` of it, grouped by row_offsets) -> (codes uint8 [K, P], scales
    float32 [P / 128, K]), transposed, one scale per 128 rows; P = mx_b128_padded_rows(R, E)."""
    M, K = _input(x)
    R = _row_index(index, x, M)
    E = 1 if row_offsets is None else _offsets(row_offsets, x)
    P = mx_b128_padded_rows(R, E)
    codes = _output(codes, "codes", (K, P), torch.uint8, x, stream)
    scales = _output(scales, "scales", (P // BLOCK128, K), torch.float32, x, stream)
    _check(lib().mx_quantize_b128_cols(_ptr(x), M, K, _ptr(index), R, _ptr(row_offsets), E,
                                       _ptr(codes), _ptr(scales), _stream_ptr(stream, x)))
    return codes, scales


def mx_quantize_b128_blocks(x, *, transpose: bool = False, codes=None, scales=None, codes_t=None,
                            scales_t=None, stream=None):
    """bf16 [M, K] or [batch, M, K] -> (codes uint8 like x, scales float32 [.., ceil(M / 128),
    ceil(K / 128)]), one scale per 128 x 128 square; with transpose also the transposed operand."""
    _tensor(x, "x", torch.bfloat16, dim=(2, 3))
    lead, (M, K) = tuple(x.shape[:-2]), x.shape[-2:]
    mb, kb = -(-M // BLOCK128), -(-K // BLOCK128)
    codes = _output(codes, "codes", (*lead, M, K), torch.uint8, x, stream)
    scales = _output(scales, "scales", (*lead, mb, kb), torch.float32, x, stream)
    if transpose:
        codes_t = _output(codes_t, "codes_t", (*lead, K, M), torch.uint8, x, stream)
        scales_t = _output(scales_t, "scales_t", (*lead, kb, mb), torch.float32, x, stream)
    else:
        codes_t = scales_t = None
    _check(lib().mx_quantize_b128_blocks(_ptr(x), lead[0] if lead else 1, M, K, _ptr(codes),
                                         _ptr(scales), _ptr(codes_t), _ptr(scales_t),
                                         _stream_ptr(stream, x)))
    return (codes, scales, codes_t, scales_t) if transpose else (codes, scales)


def _b128_operand(codes, scales, what, rows, dim=2, like=None):
    """Checks an operand whose scales are in the rows or the blocks form; returns the codes' shape."""
    _tensor(codes, f"{what}_codes", torch.uint8, dim=dim, like=like)
    _tensor(scales, f"{what}_scales", torch.float32, like=codes)
    shape = codes.shape
    R, K = shape[-2:] if dim == 3 else shape
    kb = -(-K // BLOCK128)
    want = (kb, R) if rows else (-(-R // BLOCK128), kb)
    if scales.shape != ((shape[0], *want) if dim == 3 else want):
        raise ValueError(f"{what}_scales must be {[*shape[:-2], *want]}")
    return shape


def _b128_dense(a_codes, a_scales, b_codes, b_scales, b_form):
    M, K = _b128_operand(a_codes, a_scales, "a", True)
    N, Kb = _b128_operand(b_codes, b_scales, "b", b_form == B128_ROWS, like=a_codes)
    if K != Kb:
        raise ValueError("a_codes and b_codes must be [M, K] and [N, K]")
    return M, N, K


def _out_type(out_dtype, c):
    dtype = out_dtype if c is None else c.dtype
    if dtype not in _TYPES:
        raise TypeError("the product's type is torch.bfloat16 or torch.float32")
    return dtype


def mx_gemm_b128(a_codes, a_scales, b_codes, b_scales, b_form=B128_BLOCKS, *,
                 out_dtype=torch.bfloat16, c=None, stream=None):
    """C[M, N] = A @ B^T from E4M3 codes [M, K] and [N, K] with a scale per block of 128: A's in the
    rows form, B's in the blocks form or (B128_ROWS) the rows form."""
    M, N, K = _b128_dense(a_codes, a_scales, b_codes, b_scales, b_form)
    dtype = _out_type(out_dtype, c)
    c = _output(c, "c", (M, N), dtype, a_codes, stream)
    _check(lib().mx_gemm_b128(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), M, N, K,
                              b_form, _TYPES[dtype], _ptr(c), _stream_ptr(stream, a_codes)))
    return c


def mx_selftest_gemm_b128_give_up(a_codes, a_scales, b_codes, b_scales, limit_ns: int,
                                  b_form=B128_BLOCKS, *, stream=None):
    """mx_gemm_b128 with every pipeline wait of the kernel limited to limit_ns; returns the
    (unspecified) C buffer. The device error word reports the give-up."""
    M, N, K = _b128_dense(a_codes, a_scales, b_codes, b_scales, b_form)
    c = _output(None, "c", (M, N), torch.bfloat16, a_codes, stream)
    _check(lib().mx_selftest_gemm_b128_give_up(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes),
                                               _ptr(b_scales), M, N, K, b_form, _ptr(c), limit_ns,
                                               _stream_ptr(stream, a_codes)))
    return c


def _b128_grouped(a_codes, a_scales, b_codes, b_scales, row_offsets):
    R, K = _b128_operand(a_codes, a_scales, "a", True)
    experts, N, Kb = _b128_operand(b_codes, b_scales, "b", False, 3, a_codes)
    E = _offsets(row_offsets, a_codes)
    if experts != E or K != Kb:
        raise ValueError("a_codes and b_codes must be [R, K] and [E, N, K]")
    return E, R, N, K


def mx_gemm_b128_grouped(a_codes, a_scales, b_codes, b_scales, row_offsets, *,
                         out_dtype=torch.bfloat16, c=None, stream=None):
    """Rows of A [R, K] by expert (row_offsets int64 [E + 1]) times that expert's B [E, N, K] ->
    C [R, N]; rows from row_offsets[E] on are not written."""
    E, R, N, K = _b128_grouped(a_codes, a_scales, b_codes, b_scales, row_offsets)
    dtype = _out_type(out_dtype, c)
    c = _output(c, "c", (R, N), dtype, a_codes, stream)
    _check(lib().mx_gemm_b128_grouped(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales),
                                      _ptr(row_offsets), E, R, N, K, _TYPES[dtype], _ptr(c),
                                      _stream_ptr(stream, a_codes)))
    return c


def mx_selftest_gemm_b128_grouped_give_up(a_codes, a_scales, b_codes, b_scales, row_offsets,
                                          limit_ns: int, *, stream=None):
    """mx_gemm_b128_grouped with every pipeline wait of the kernel limited to limit_ns; returns the
    (unspecified) C buffer. The device error word reports the give-up."""
    E, R, N, K = _b128_grouped(a_codes, a_scales, b_codes, b_scales, row_offsets)
    c = _output(None, "c", (R, N), torch.bfloat16, a_codes, stream)
    _check(lib().mx_selftest_gemm_b128_grouped_give_up(
        _ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), _ptr(row_offsets), E, R, N, K,
        _ptr(c), limit_ns, _stream_ptr(stream, a_codes)))
    return c


def mx_gemm_b128_grouped_wgrad(a_codes, a_scales, b_codes, b_scales, row_offsets, *,
                               out_dtype=torch.float32, c=None, stream=None):
    """C[e] = A_e @ B_e^T over expert e's rows, from mx_quantize_b128_cols operands [M, P] and
    [N, P] of the same row_offsets -> C [E, M, N]."""
    M, P = _b128_operand(a_codes, a_scales, "a", True)
    N, Pb = _b128_operand(b_codes, b_scales, "b", True, like=a_codes)
    E = _offsets(row_offsets, a_codes)
    if P != Pb:
        raise ValueError("a_codes and b_codes must be [M, P] and [N, P]")
    dtype = _out_type(out_dtype, c)
    c = _output(c, "c", (E, M, N), dtype, a_codes, stream)
    _check(lib().mx_gemm_b128_grouped_wgrad(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes),
                                            _ptr(b_scales), _ptr(row_offsets), E, M, N, P,
                                            _TYPES[dtype], _ptr(c), _stream_ptr(stream, a_codes)))
    return c


def _slots(y, slots, weights):
    _input(y, "y")
    _tensor(slots, "slots", torch.int32, dim=2, like=y)
    if weights is not None and \
            _tensor(weights, "weights", torch.float32, like=y).shape != slots.shape:
        raise ValueError("weights must be [T, k] as slots")
    return slots.shape


def mx_combine(y, slots, weights=None, *, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * y[slots[t, j]]: bf16 rows [R, N] -> [T, N] (weights None: ones)."""
    T, k = _slots(y, slots, weights)
    R, N = y.shape
    out = _output(out, "out", (T, N), torch.bfloat16, y, stream)
    _check(lib().mx_combine(_ptr(y), _ptr(slots), _ptr(weights), T, k, R, N, _ptr(out),
                            _stream_ptr(stream, y)))
    return out


def mx_combine_backward(dout, y, slots, weights, *, dy=None, dweights=None, stream=None):
    """Gradients of mx_combine: dout [T, N] -> (dy [R, N], dweights [T, k]). Rows of dy that no slot names
    are zeros; in a dy that is passed they keep what they held."""
    T, k = _slots(y, slots, weights)
    R, N = y.shape
    if _tensor(dout, "dout", torch.bfloat16, dim=2, like=y).shape != (T, N):
        raise ValueError("dout must be [T, N]")
    dweights = _output(dweights, "dweights", (T, k), torch.float32, y, stream)
    if dy is None:
        dy = _empty((R, N), torch.bfloat16, y, stream)
        workspace = _empty((R,), torch.int32, y, stream, scratch=True)
        _check(lib().mx_combine_backward_whole(_ptr(dout), _ptr(y), _ptr(slots), _ptr(weights), T, k, R,
                                               N, _ptr(dy), _ptr(dweights), _ptr(workspace),
                                               _stream_ptr(stream, y)))
    else:
        _output(dy, "dy", (R, N), torch.bfloat16, y, stream)
        _check(lib().mx_combine_backward(_ptr(dout), _ptr(y), _ptr(slots), _ptr(weights), T, k, R, N,
                                         _ptr(dy), _ptr(dweights), _stream_ptr(stream, y)))
    return dy, dweights
