"""Python binding of ``libi8ql.so`` (argument marshalling only).

Each function keeps the name of its C entry point, takes torch CUDA tensors,
checks dtypes, shapes and contiguity, allocates any output the caller did not
pass (torch is only the device-memory and stream provider), and calls the C
ABI with raw device pointers and the current CUDA stream.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback.  If the
library is missing, loading fails with an error that says how to build it.

Calls run on torch's current stream, or on `stream` (a torch stream or a raw
handle); what a call allocates itself belongs to that stream, as if the stream
had been current.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libi8ql.so")

I8QL_OK = 0
I8QL_ERR_INVALID_ARG = 1
I8QL_ERR_UNSUPPORTED = 2
I8QL_ERR_CUDA = 3
I8QL_ERR_TIMEOUT = 4
I8QL_ERR_BAD_OFFSETS = 5
I8QL_ERR_NO_DEVICE = 6
I8QL_ERR_WORKSPACE_LIMIT = 7
I8QL_ERR_BAD_INDEX = 8
I8QL_MAX_K = 133144
I8QL_NOALLOC_MAX_ELEMENTS = 16 * 1024 * 1024
I8QL_KV_MIN_PAGE = 16
I8QL_KV_MAX_PAGE = 256
I8QL_ROTARY_MAX_D = 512
I8QL_W8A8_DECODE_MAX_M = 32  # w8a8_gemm runs the decode kernel up to this M

# Every symbol the C header declares, with its ctypes signature.
_P, _I64, _S, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
SIGNATURES = {
    "quantize_weight_per_channel_int8": (_S, [_P, _I64, _I64, _P, _P, _P]),
    "quantize_act_per_token_int8": (_S, [_P, _I64, _I64, _P, _P, _P]),
    "w8a8_gemm": (_S, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w8a8_gemm_noalloc": (_S, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w8a8_linear": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w8a16_gemm": (_S, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "grouped_w8a16_gemm": (_S, [_P, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _P]),
    "i8ql_w8a8_plan": (_S, [_I64, _I64, _I64, _P, _P, _P]),
    "i8ql_fp8_plan": (_S, [_I64, _I64, _I64, _P, _P, _P]),
    "i8ql_w8a8_noalloc_plan": (_S, [_I64, _I64, _I64, _P, _P, _P]),
    "i8ql_w8a8_linear_launches": (_S, [_I64, _I64, _I64, _P]),
    "i8ql_get_device_error": (_S, [_P]),
    "i8ql_status_string": (ctypes.c_char_p, [_S]),
    "i8ql_version": (_S, []),
    "i8ql_debug_stream_k_timeout": (None, [_S]),
    "i8ql_set_early_weight_loads": (None, [_S]),
    "i8ql_early_weight_loads": (_S, []),
    "quantize_weight_per_channel_fp8": (_S, [_P, _I64, _I64, _P, _P, _P]),
    "quantize_act_per_token_fp8": (_S, [_P, _I64, _I64, _P, _P, _P]),
    "w8a8_fp8_gemm": (_S, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w8a8_fp8_linear": (_S, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "quantize_weight_w4_g128": (_S, [_P, _I64, _I64, _P, _P, _P]),
    "w4a16_gemm": (_S, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w8a8_linear_fused": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "moe_route_topk": (_S, [_P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "grouped_w8a16_silu_mul": (_S, [_P, _P, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _P]),
    "moe_combine": (_S, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "kv_cache_store": (_S, [_P, _P, _I64, _I64, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P]),
    "kv_cache_load": (_S, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P]),
    "kv_cache_attention": (_S, [_P, _I64, _P, _P, _P, _I64, _P, _P, _P, *[_I64] * 10, _F, _P, _I64, _P]),
    "i8ql_kv_attention_workspace": (_S, [*[_I64] * 9, _P]),
    "rotary_table": (_S, [_P, _P, _P, _I64, _I64, _F, _P]),
    "rotary_apply": (_S, [_P, _I64, _P, _I64, _P, _P, *[_I64] * 5, _S, _S, _P]),
    "kv_cache_store_rotary": (_S, [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P, *[_I64] * 8, _S, _P]),
    "kv_cache_weights": (_S, [_P, _I64, _P, _P, _P, _I64, _P, _P, _P, _P, *[_I64] * 10, _F, _P, _I64, _P]),
    "i8ql_kv_weights_workspace": (_S, [*[_I64] * 9, _P]),
    "kv_cache_evict": (_S, [_P, _P, _P, _P, _I64, _P, _P, _I64, _P, _P, *[_I64] * 9, _P]),
    "moe_expert_mlp_w8a16": (_S, [_P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
}

_LIB = None


class I8qlError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIBRARY):
            raise ImportError(
                f"{LIBRARY} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        handle = ctypes.CDLL(LIBRARY)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def status_string(status: int) -> str:
    return lib().i8ql_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != I8QL_OK:
        raise I8qlError(status, where)


def _stream(stream) -> int | None:
    if stream is None:
        if torch.cuda.is_initialized():  # the same handle without a Stream object (2.9 -> 0.3 us a call)
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(shape: tuple, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """torch.empty with the call's stream current, so that the allocator knows
    which stream uses the memory (and does not hand out a block that the
    current stream has freed but may still be reading)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        # (0 is the default stream's handle; ExternalStream makes a new stream of it)
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str, device: int | None = None) -> None:
    """Checks a dense CUDA tensor; with `device`, that it is on that one (its index)."""
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and (
            t.is_cuda if device is None else t.get_device() == device) and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.numel() and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.numel() and device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the cache's device (cuda:{device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _quant(fn_name: str, src: torch.Tensor, q, scale, stream):
    if src.dim() != 2:
        raise ValueError("input must be 2-D [rows, K]")
    rows, k = src.shape
    _need(src, torch.bfloat16, (rows, k), "input")
    if q is None:
        q = _empty((rows, k), torch.int8, src.device, stream)
    if scale is None:
        scale = _empty((rows,), torch.float32, src.device, stream)
    _need(q, torch.int8, (rows, k), "q")
    _need(scale, torch.float32, (rows,), "scale")
    st = getattr(lib(), fn_name)(_ptr(src), rows, k, _ptr(q), _ptr(scale), _stream(stream))
    _check(st, fn_name)
    return q, scale


def quantize_weight_per_channel_int8(w: torch.Tensor, q=None, scale=None, stream=None):
    """int8 codes [N, K] and fp32 per-output-channel scales [N] of bf16 w."""
    return _quant("quantize_weight_per_channel_int8", w, q, scale, stream)


def quantize_act_per_token_int8(x: torch.Tensor, q=None, scale=None, stream=None):
    """int8 codes [M, K] and fp32 per-token scales [M] of bf16 x."""
    return _quant("quantize_act_per_token_int8", x, q, scale, stream)


def w8a8_linear(x, qw, sw, bias=None, y=None, qx=None, sx=None, acc_debug=None, stream=None, fused=False):
    """bf16 y [M, N] = w8a8_gemm(quantize_act_per_token_int8(x), qw, sw, bias),
    with the quantization fused into the call; qx / sx, when given, receive
    the token codes and scales.  fused=True takes the one-launch entry point
    (w8a8_linear_fused, M <= 8)."""
    m, k = x.shape
    n = qw.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(qw, torch.int8, (n, k), "qw")
    _need(sw, torch.float32, (n,), "sw")
    if bias is not None:
        _need(bias, torch.bfloat16, (n,), "bias")
    if y is None:
        y = _empty((m, n), torch.bfloat16, qw.device, stream)
    _need(y, torch.bfloat16, (m, n), "y")
    if qx is not None:
        _need(qx, torch.int8, (m, k), "qx")
    if sx is not None:
        _need(sx, torch.float32, (m,), "sx")
    if acc_debug is not None:
        _need(acc_debug, torch.int32, (m, n), "acc_debug")
    name = "w8a8_linear_fused" if fused else "w8a8_linear"
    st = getattr(lib(), name)(_ptr(x), _ptr(qw), _ptr(sw), _ptr(bias), _ptr(y), _ptr(qx), _ptr(sx),
                              _ptr(acc_debug), m, n, k, _stream(stream))
    _check(st, name)
    return y


def w8a8_gemm(qx, sx, qw, sw, bias=None, y=None, acc_debug=None, stream=None):
    """bf16 y [M, N] = ((float)(qx @ qw^T) * sx[:, None]) * sw[None, :] (+ bias)."""
    m, k = qx.shape
    n = qw.shape[0]
    _need(qx, torch.int8, (m, k), "qx")
    _need(sx, torch.float32, (m,), "sx")
    _need(qw, torch.int8, (n, k), "qw")
    _need(sw, torch.float32, (n,), "sw")
    if bias is not None:
        _need(bias, torch.bfloat16, (n,), "bias")
    if y is None:
        y = _empty((m, n), torch.bfloat16, qw.device, stream)
    _need(y, torch.bfloat16, (m, n), "y")
    if acc_debug is not None:
        _need(acc_debug, torch.int32, (m, n), "acc_debug")
    st = lib().w8a8_gemm(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(bias), _ptr(y),
                         _ptr(acc_debug), m, n, k, _stream(stream))
    _check(st, "w8a8_gemm")
    return y


def w8a8_gemm_noalloc(qx, sx, qw, sw, y, bias=None, acc_debug=None, stream=None):
    """w8a8_gemm through the entry point that allocates no device memory.

    For callers that cannot allocate while they run (graph replay with fixed
    memory, allocator-free serving loops): the output ``y`` must be passed in,
    and the large-M workspace comes from a fixed array inside the library, so
    ``M * K`` may not exceed ``I8QL_NOALLOC_MAX_ELEMENTS`` when M > 32.
    Calls that could overlap on the GPU must not be issued (they share it).
    """
    m, k = qx.shape
    n = qw.shape[0]
    _need(qx, torch.int8, (m, k), "qx")
    _need(sx, torch.float32, (m,), "sx")
    _need(qw, torch.int8, (n, k), "qw")
    _need(sw, torch.float32, (n,), "sw")
    _need(y, torch.bfloat16, (m, n), "y")
    if bias is not None:
        _need(bias, torch.bfloat16, (n,), "bias")
    if acc_debug is not None:
        _need(acc_debug, torch.int32, (m, n), "acc_debug")
    st = lib().w8a8_gemm_noalloc(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(bias), _ptr(y),
                                 _ptr(acc_debug), m, n, k, _stream(stream))
    _check(st, "w8a8_gemm_noalloc")
    return y


def w8a16_gemm(x, qw, sw, y=None, stream=None):
    """bf16 y [M, N] = bf16(sw[n] * sum_k qw[n, k] * x[m, k])."""
    m, k = x.shape
    n = qw.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(qw, torch.int8, (n, k), "qw")
    _need(sw, torch.float32, (n,), "sw")
    if y is None:
        y = _empty((m, n), torch.bfloat16, qw.device, stream)
    _need(y, torch.bfloat16, (m, n), "y")
    st = lib().w8a16_gemm(_ptr(x), _ptr(qw), _ptr(sw), _ptr(y), m, n, k, _stream(stream))
    _check(st, "w8a16_gemm")
    return y


def grouped_w8a16_gemm(x, offsets, qw, sw, y=None, stream=None):
    """Grouped W8A16: rows offsets[e] .. offsets[e+1] of x use expert e."""
    t, k = x.shape
    e, n, k2 = qw.shape
    if k2 != k:
        raise ValueError("qw and x disagree on K")
    _need(x, torch.bfloat16, (t, k), "x")
    _need(offsets, torch.int32, (e + 1,), "offsets")
    _need(qw, torch.int8, (e, n, k), "qw")
    _need(sw, torch.float32, (e, n), "sw")
    if y is None:
        y = _empty((t, n), torch.bfloat16, qw.device, stream)
    _need(y, torch.bfloat16, (t, n), "y")
    st = lib().grouped_w8a16_gemm(_ptr(x), _ptr(offsets), e, _ptr(qw), _ptr(sw), _ptr(y), t, n, k,
                                  _stream(stream))
    _check(st, "grouped_w8a16_gemm")
    return y


def _plan(fn_name: str, m: int, n: int, k: int) -> tuple[int, int, int]:
    tile_n, split_k, pair = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
    _check(getattr(lib(), fn_name)(m, n, k, ctypes.byref(tile_n), ctypes.byref(split_k), ctypes.byref(pair)),
           fn_name)
    return tile_n.value, split_k.value, pair.value


def i8ql_w8a8_plan(m: int, n: int, k: int) -> tuple[int, int, int]:
    """(tile width, split-K factor, CTA-pair mode: 0 single CTAs, 1 pairs,
    2 pairs with stream-K) w8a8_gemm uses for an M x N x K problem on the
    current device; (0, 0, 0) in the decode range (M <= I8QL_W8A8_DECODE_MAX_M)."""
    return _plan("i8ql_w8a8_plan", m, n, k)


def i8ql_fp8_plan(m: int, n: int, k: int) -> tuple[int, int, int]:
    """(tile width, split-K factor, CTA pairs 0/1) w8a8_fp8_gemm uses for an
    M x N x K problem on the current device."""
    return _plan("i8ql_fp8_plan", m, n, k)


def i8ql_w8a8_noalloc_plan(m: int, n: int, k: int) -> tuple[int, int, int]:
    """The same for w8a8_gemm_noalloc (never stream-K)."""
    return _plan("i8ql_w8a8_noalloc_plan", m, n, k)


def i8ql_w8a8_linear_launches(m: int, n: int, k: int) -> int:
    """Kernels one w8a8_linear call of this size launches on the current
    device: 1 with the quantization inside the decode GEMM, else 2 (0 for
    m == 0)."""
    launches = ctypes.c_int32(-1)
    _check(lib().i8ql_w8a8_linear_launches(m, n, k, ctypes.byref(launches)), "i8ql_w8a8_linear_launches")
    return launches.value


def i8ql_get_device_error(stream=None) -> int:
    """Wait for the stream, then read and clear the sticky kernel-fault word."""
    return int(lib().i8ql_get_device_error(_stream(stream)))


def i8ql_version() -> int:
    return int(lib().i8ql_version())


def i8ql_debug_stream_k_timeout(on: bool) -> None:
    """Test hook: while on, stream-K finishers wait for a flag nothing writes
    (1 ms limit), so the call records I8QL_ERR_TIMEOUT without hanging."""
    lib().i8ql_debug_stream_k_timeout(1 if on else 0)


def i8ql_set_early_weight_loads(on: bool) -> None:
    """Serving option: decode-size GEMMs load their first weights before
    waiting for the previous kernel on the stream (which must not write
    them).  Process-wide; off by default."""
    lib().i8ql_set_early_weight_loads(1 if on else 0)


def i8ql_early_weight_loads() -> bool:
    return bool(lib().i8ql_early_weight_loads())


# ---------------------------------------------------------------- FP8 E4M3

def _quant_fp8(fn_name: str, src: torch.Tensor, q, scale, stream):
    if src.dim() != 2:
        raise ValueError("input must be 2-D [rows, K]")
    rows, k = src.shape
    _need(src, torch.bfloat16, (rows, k), "input")
    if q is None:
        q = _empty((rows, k), torch.uint8, src.device, stream)
    if scale is None:
        scale = _empty((rows,), torch.float32, src.device, stream)
    _need(q, torch.uint8, (rows, k), "q")
    _need(scale, torch.float32, (rows,), "scale")
    _check(getattr(lib(), fn_name)(_ptr(src), rows, k, _ptr(q), _ptr(scale), _stream(stream)), fn_name)
    return q, scale


def quantize_weight_per_channel_fp8(w: torch.Tensor, q=None, scale=None, stream=None):
    """E4M3 codes [N, K] (uint8) and fp32 per-channel scales (absmax / 448)."""
    return _quant_fp8("quantize_weight_per_channel_fp8", w, q, scale, stream)


def quantize_act_per_token_fp8(x: torch.Tensor, q=None, scale=None, stream=None):
    """E4M3 codes [M, K] (uint8) and fp32 per-token scales (absmax / 448)."""
    return _quant_fp8("quantize_act_per_token_fp8", x, q, scale, stream)


def w8a8_fp8_gemm(qx, sx, qw, sw, bias=None, y=None, stream=None):
    """bf16 y [M, N] = ((sum_k e4m3(qx) e4m3(qw)) * sx[:, None]) * sw[None, :] (+ bias)."""
    m, k = qx.shape
    n = qw.shape[0]
    _need(qx, torch.uint8, (m, k), "qx")
    _need(sx, torch.float32, (m,), "sx")
    _need(qw, torch.uint8, (n, k), "qw")
    _need(sw, torch.float32, (n,), "sw")
    if bias is not None:
        _need(bias, torch.bfloat16, (n,), "bias")
    if y is None:
        y = _empty((m, n), torch.bfloat16, qw.device, stream)
    _need(y, torch.bfloat16, (m, n), "y")
    _check(lib().w8a8_fp8_gemm(_ptr(qx), _ptr(sx), _ptr(qw), _ptr(sw), _ptr(bias), _ptr(y), m, n, k,
                               _stream(stream)), "w8a8_fp8_gemm")
    return y


def w8a8_fp8_linear(x, qw, sw, bias=None, y=None, qx=None, sx=None, stream=None):
    """bf16 y = w8a8_fp8_gemm(quantize_act_per_token_fp8(x), qw, sw, bias) in one call."""
    m, k = x.shape
    n = qw.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(qw, torch.uint8, (n, k), "qw")
    _need(sw, torch.float32, (n,), "sw")
    if bias is not None:
        _need(bias, torch.bfloat16, (n,), "bias")
    if y is None:
        y = _empty((m, n), torch.bfloat16, qw.device, stream)
    _need(y, torch.bfloat16, (m, n), "y")
    if qx is not None:
        _need(qx, torch.uint8, (m, k), "qx")
    if sx is not None:
        _need(sx, torch.float32, (m,), "sx")
    _check(lib().w8a8_fp8_linear(_ptr(x), _ptr(qw), _ptr(sw), _ptr(bias), _ptr(y), _ptr(qx), _ptr(sx), m, n, k,
                                 _stream(stream)), "w8a8_fp8_linear")
    return y


# ---------------------------------------------------------------- W4A16, group 128

def quantize_weight_w4_g128(w: torch.Tensor, q=None, scale=None, stream=None):
    """Packed int4 codes [N, K/2] (uint8) and bf16 group scales [N, K/128]."""
    n, k = w.shape
    _need(w, torch.bfloat16, (n, k), "w")
    if q is None:
        q = _empty((n, k // 2), torch.uint8, w.device, stream)
    if scale is None:
        scale = _empty((n, k // 128), torch.bfloat16, w.device, stream)
    _need(q, torch.uint8, (n, k // 2), "q")
    _need(scale, torch.bfloat16, (n, k // 128), "scale")
    _check(lib().quantize_weight_w4_g128(_ptr(w), n, k, _ptr(q), _ptr(scale), _stream(stream)),
           "quantize_weight_w4_g128")
    return q, scale


def w4a16_gemm(x, q, scale, y=None, stream=None):
    """bf16 y [M, N] = bf16(sum_g scale[n, g] * sum_k q[n, k] * x[m, k])."""
    m, k = x.shape
    n = q.shape[0]
    _need(x, torch.bfloat16, (m, k), "x")
    _need(q, torch.uint8, (n, k // 2), "q")
    _need(scale, torch.bfloat16, (n, k // 128), "scale")
    if y is None:
        y = _empty((m, n), torch.bfloat16, q.device, stream)
    _need(y, torch.bfloat16, (m, n), "y")
    _check(lib().w4a16_gemm(_ptr(x), _ptr(q), _ptr(scale), _ptr(y), m, n, k, _stream(stream)), "w4a16_gemm")
    return y


# ---------------------------------------------------------------- MoE expert MLP

def moe_route_topk(logits, top_k, n_shared, stream=None):
    """Device routing: (offsets [E+n_shared+1], row_token [T*S], token_row
    [T, S], slot_weight [T, S]) for fp32 logits [T, E]."""
    t, e = logits.shape
    _need(logits, torch.float32, (t, e), "logits")
    s = top_k + n_shared
    dev = logits.device
    offsets = _empty((e + n_shared + 1,), torch.int32, dev, stream)
    row_token = _empty((t * s,), torch.int32, dev, stream)
    token_row = _empty((t, s), torch.int32, dev, stream)
    slot_weight = _empty((t, s), torch.float32, dev, stream)
    _check(lib().moe_route_topk(_ptr(logits), t, e, top_k, n_shared, _ptr(offsets), _ptr(row_token),
                                _ptr(token_row), _ptr(slot_weight), _stream(stream)), "moe_route_topk")
    return offsets, row_token, token_row, slot_weight


def grouped_w8a16_silu_mul(x, row_token, offsets, qw, sw, h=None, rows=None, stream=None):
    """h [rows, I] = bf16(silu(gate) * up) of the grouped fused gate/up
    projection qw [E, 2I, K], gathering token rows through row_token."""
    e, two_i, k = qw.shape
    inter = two_i // 2
    if rows is None:
        rows = row_token.shape[0] if row_token is not None else x.shape[0]
    _need(x, torch.bfloat16, (x.shape[0], k), "x")
    _need(offsets, torch.int32, (e + 1,), "offsets")
    if row_token is not None:
        _need(row_token, torch.int32, (rows,), "row_token")
    _need(sw, torch.float32, (e, two_i), "sw")
    if h is None:
        h = _empty((rows, inter), torch.bfloat16, qw.device, stream)
    _need(h, torch.bfloat16, (rows, inter), "h")
    _check(lib().grouped_w8a16_silu_mul(_ptr(x), _ptr(row_token), _ptr(offsets), e, _ptr(qw), _ptr(sw), _ptr(h),
                                        rows, inter, k, _stream(stream)), "grouped_w8a16_silu_mul")
    return h


def moe_combine(yd, token_row, slot_weight, out=None, stream=None):
    """out [T, H] = bf16(sum_s slot_weight[t, s] * yd[token_row[t, s]])."""
    t, s = token_row.shape
    h = yd.shape[1]
    _need(token_row, torch.int32, (t, s), "token_row")
    _need(slot_weight, torch.float32, (t, s), "slot_weight")
    _need(yd, torch.bfloat16, (yd.shape[0], h), "yd")
    if out is None:
        out = _empty((t, h), torch.bfloat16, yd.device, stream)
    _need(out, torch.bfloat16, (t, h), "out")
    _check(lib().moe_combine(_ptr(yd), _ptr(token_row), _ptr(slot_weight), _ptr(out), t, s, h, _stream(stream)),
           "moe_combine")
    return out


def moe_expert_mlp_w8a16(x, logits, top_k, n_shared, qw_gate_up, sw_gate_up, qw_down, sw_down, out=None,
                         stream=None):
    """The MoE expert MLP end to end (routing, gate/up + SiLU gate, down,
    combine) for tokens x [T, H] with gate logits [T, E_routed]."""
    t, hid = x.shape
    e_r = logits.shape[1]
    e, two_i, k = qw_gate_up.shape
    inter = two_i // 2
    _need(x, torch.bfloat16, (t, hid), "x")
    _need(logits, torch.float32, (t, e_r), "logits")
    if e != e_r + n_shared or k != hid:
        raise ValueError("expert weights do not match the routing or the hidden size")
    _need(qw_gate_up, torch.int8, (e, two_i, hid), "qw_gate_up")
    _need(sw_gate_up, torch.float32, (e, two_i), "sw_gate_up")
    _need(qw_down, torch.int8, (e, hid, inter), "qw_down")
    _need(sw_down, torch.float32, (e, hid), "sw_down")
    if out is None:
        out = _empty((t, hid), torch.bfloat16, x.device, stream)
    _need(out, torch.bfloat16, (t, hid), "out")
    _check(lib().moe_expert_mlp_w8a16(_ptr(x), _ptr(logits), e_r, top_k, n_shared, _ptr(qw_gate_up),
                                      _ptr(sw_gate_up), _ptr(qw_down), _ptr(sw_down), _ptr(out), t, hid, inter,
                                      _stream(stream)), "moe_expert_mlp_w8a16")
    return out


# ---------------------------------------------------------------- quantized key/value cache

def kv_cache_alloc(num_pages, heads, page_size, head_dim, bits=4, device="cuda"):
    """An empty cache of num_pages pages: codes uint8 [num_pages, 2, heads,
    page_size, head_dim * bits / 8] and params bf16 [num_pages, 2, heads,
    page_size, 2] (scale, low); index 0 of the second axis holds the keys."""
    if bits not in (4, 8):
        raise ValueError("bits must be 4 or 8")
    codes = torch.empty((num_pages, 2, heads, page_size, head_dim * bits // 8), dtype=torch.uint8, device=device)
    params = torch.empty((num_pages, 2, heads, page_size, 2), dtype=torch.bfloat16, device=device)
    return codes, params


def _kv_cache(codes: torch.Tensor, params: torch.Tensor, head_dim: int) -> tuple[int, int, int, int, int | None]:
    """(num_pages, heads, page_size, bits, device index) of a cache for rows of
    head_dim channels, which has to be on the current device."""
    shape = codes.shape
    if len(shape) != 5 or shape[1] != 2:
        raise ValueError("codes must be [num_pages, 2, heads, page_size, head_dim * bits / 8]")
    pages, _, heads, page, row = shape
    bits = 4 if 2 * row == head_dim else 8
    _need(codes, torch.uint8, (pages, 2, heads, page, head_dim * bits // 8), "codes")
    device = codes.get_device() if codes.is_cuda else None
    if device is not None and device != torch._C._cuda_getDevice():
        raise ValueError(f"codes is on {codes.device}, not on the current device (cuda:{torch.cuda.current_device()})")
    _need(params, torch.bfloat16, (pages, 2, heads, page, 2), "params", device)
    return pages, heads, page, bits, device


def _need_heads(t: torch.Tensor, heads: int, head_dim: int, name: str, device: int | None) -> int:
    """Checks bf16 [T, heads, head_dim] whose tokens are dense (tokens may lie
    apart: a slice of a fused projection's rows), on the cache's device;
    returns their distance."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim:
        raise ValueError(f"{name} must have shape [T, {heads}, {head_dim}], got {tuple(shape)}")
    tokens = shape[0]
    if t.get_device() != device and t.numel():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} is on {t.device}, not on the cache's device (cuda:{device})")
    if tokens <= 1 and t.is_contiguous():
        return heads * head_dim
    step, head_step, one = t.stride()
    if tokens and (one != 1 or (head_step != head_dim and heads > 1)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return step if tokens > 1 else heads * head_dim


def kv_cache_store(k, v, slots, codes, params, stream=None):
    """Quantizes keys and values, bf16 [T, heads, head_dim] (slices of a fused
    projection are fine), into the cache rows slots (int64 [T]: page *
    page_size + place; negative: skipped).  Returns (codes, params)."""
    if k.dim() != 3:
        raise ValueError("k must be [T, heads, head_dim]")
    t, h, d = k.shape
    pages, heads, page, bits, device = _kv_cache(codes, params, d)
    k_step = _need_heads(k, heads, d, "k", device)
    v_step = _need_heads(v, heads, d, "v", device)
    if v.shape[0] != t:
        raise ValueError("k and v disagree on T")
    _need(slots, torch.int64, (t,), "slots", device)
    st = lib().kv_cache_store(k.data_ptr(), v.data_ptr(), k_step, v_step, slots.data_ptr(), codes.data_ptr(),
                              params.data_ptr(), t, h, d, bits, page, pages, _stream(stream))
    if st != I8QL_OK:
        _check(st, "kv_cache_store")
    return codes, params


def kv_cache_load(codes, params, slots, head_dim, k=None, v=None, stream=None):
    """(k, v) bf16 [T, heads, head_dim]: the cache rows at slots, bf16(low +
    scale * code); zeros where the slot is negative."""
    pages, heads, page, bits, device = _kv_cache(codes, params, head_dim)
    t = slots.shape[0]
    _need(slots, torch.int64, (t,), "slots", device)
    shape = (t, heads, head_dim)
    if k is None:
        k = _empty(shape, torch.bfloat16, codes.device, stream)
    else:
        _need(k, torch.bfloat16, shape, "k", device)
    if v is None:
        v = _empty(shape, torch.bfloat16, codes.device, stream)
    else:
        _need(v, torch.bfloat16, shape, "v", device)
    st = lib().kv_cache_load(codes.data_ptr(), params.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr(), t,
                             heads, head_dim, bits, page, pages, _stream(stream))
    if st != I8QL_OK:
        _check(st, "kv_cache_load")
    return k, v


def i8ql_kv_attention_workspace(batch, tokens, q_heads, heads, head_dim, bits, page_size, table_width, max_q=1) -> int:
    """Bytes of workspace a kv_cache_attention call of these sizes takes on
    the current device."""
    n = ctypes.c_int64(0)
    _check(lib().i8ql_kv_attention_workspace(batch, tokens, q_heads, heads, head_dim, bits, page_size, table_width,
                                             max_q, ctypes.byref(n)), "i8ql_kv_attention_workspace")
    return n.value


@functools.lru_cache(maxsize=1024)
def _workspace_size(device: int, *sizes) -> int:
    """The same, asked once per device and sizes (a function of those alone)."""
    return i8ql_kv_attention_workspace(*sizes)


def kv_cache_attention(q, codes, params, page_table, kv_lens, q_offsets=None, max_q=None, window=0, scale=None,
                       out=None, workspace=None, stream=None):
    """Causal attention of bf16 q [T, q_heads, head_dim] over the cache.

    Sequence b has kv_lens[b] (int32 [B]) tokens in the pages page_table[b]
    (int32 [B, width]) and the query rows q_offsets[b] .. q_offsets[b+1]
    (int32 [B+1]; None: one row each), its last tokens.  max_q: an upper bound
    of one sequence's query rows, when known (it chooses the kernel).  window:
    how many tokens a query sees, itself included (0: all).  scale: the
    softmax scale, head_dim ** -0.5 by default.  workspace: uint8, at least
    i8ql_kv_attention_workspace bytes (taken from torch when None).  Returns
    bf16 [T, q_heads, head_dim]."""
    if q.dim() != 3:
        raise ValueError("q must be [T, q_heads, head_dim]")
    t, hq, d = q.shape
    pages, heads, page, bits, device = _kv_cache(codes, params, d)
    q_step = _need_heads(q, hq, d, "q", device)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, width]")
    b, width = page_table.shape
    _need(page_table, torch.int32, (b, width), "page_table", device)
    _need(kv_lens, torch.int32, (b,), "kv_lens", device)
    if q_offsets is not None:
        _need(q_offsets, torch.int32, (b + 1,), "q_offsets", device)
    if max_q is None:
        max_q = 1 if q_offsets is None else max(t, 1)
    if out is None:
        out = _empty((t, hq, d), torch.bfloat16, codes.device, stream)
    else:
        _need(out, torch.bfloat16, (t, hq, d), "out", device)
    if workspace is None:
        size = 0
        if t and b:
            size = _workspace_size(torch.cuda.current_device(), b, t, hq, heads, d, bits, page, width, max_q)
        if size:
            workspace = _empty((size,), torch.uint8, codes.device, stream)
    else:
        _need(workspace, torch.uint8, (workspace.numel(),), "workspace", device)
        size = workspace.numel()
    st = lib().kv_cache_attention(q.data_ptr(), q_step, codes.data_ptr(), params.data_ptr(), page_table.data_ptr(), width,
                                  kv_lens.data_ptr(), None if q_offsets is None else q_offsets.data_ptr(),
                                  out.data_ptr(), b, t, hq, heads, d, bits, page, pages, max_q, window,
                                  d ** -0.5 if scale is None else scale,
                                  None if workspace is None else workspace.data_ptr(), size, _stream(stream))
    if st != I8QL_OK:
        _check(st, "kv_cache_attention")
    return out


# ---------------------------------------------------------------- rotary positions

def rotary_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=0, low=1.0, high=4.0, device="cuda"):
    """fp64 [rot / 2]: radians a position of rotary channel pairs,
    base ** (-2 i / rot), scaled for contexts `factor` times as long:

    None      as they are
    "linear"  all divided by factor (positions are interpolated)
    "base"    a larger base, that divides the slowest by factor and leaves the
              fastest
    "turns"   by how often pair i turns over `original` positions,
              n = original f / 2 pi: divided by factor up to n = low, as they
              are from n = high on, between them blended linearly in n
    "index"   the same, blended linearly in i between the (whole) indices that
              turn `high` (usually 32) and `low` times, which are held to 0 and
              rot - 1: the second may lie behind the last pair
    """
    if rot <= 0 or rot % 2 or base <= 1.0 or factor < 1.0:
        raise ValueError("rot must be positive and even, base above 1, factor at least 1")
    if scaling in ("turns", "index") and not (original > 0 and 0 < low < high):
        raise ValueError("scaling by turns needs original > 0 and 0 < low < high")
    n = rot // 2
    if scaling == "base":
        if rot == 2:
            raise ValueError("a single frequency has no base to scale")
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(n)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "turns":
        keep = [min(max((original * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
        f = [x * ((1 - k) / factor + k) for x, k in zip(f, keep)]
    elif scaling == "index":
        at = lambda turns: n * math.log(original / (2 * math.pi * turns)) / math.log(base)  # noqa: E731
        begin, end = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        keep = [1 - min(max((i - begin) / max(end - begin, 1e-3), 0.0), 1.0) for i in range(n)]
        f = [x * ((1 - k) / factor + k) for x, k in zip(f, keep)]
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.tensor(f, dtype=torch.float64, device=device)


def _current(t: torch.Tensor, name: str) -> int | None:
    """The tensor's device index (None: not a CUDA tensor), which has to be the current device's."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        return None
    device = t.get_device()
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, not on the current device (cuda:{torch.cuda.current_device()})")
    return device


def rotary_table(freqs, positions, amplitude=1.0, table=None, stream=None):
    """fp32 [P, 2F]: amplitude times the cosines, then the sines, of p *
    freqs (fp64 [F], see rotary_frequencies) for the positions 0 .. P-1 (an
    int) or those of an int64 tensor [P]."""
    device = _current(freqs, "freqs")
    f = freqs.shape[0] if freqs.dim() == 1 else -1
    _need(freqs, torch.float64, (f,), "freqs", device)
    if isinstance(positions, torch.Tensor):
        p = positions.shape[0] if positions.dim() == 1 else -1
        _need(positions, torch.int64, (p,), "positions", device)
        at = positions.data_ptr()
    else:
        p, at = int(positions), None
        if p < 0:
            raise ValueError("positions must not be negative")
    if table is None:
        table = _empty((p, 2 * f), torch.float32, freqs.device, stream)
    else:
        _need(table, torch.float32, (p, 2 * f), "table", device)
    _check(lib().rotary_table(freqs.data_ptr(), at, table.data_ptr(), p, f, amplitude, _stream(stream)), "rotary_table")
    return table


def _rotary(table, positions, tokens: int, device) -> tuple[int, int, int | None]:
    """(rows, channels turned, positions' address) of a table for so many tokens."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [rows, rot]")
    _need(table, torch.float32, tuple(table.shape), "table", device)
    if positions is None:
        return table.shape[0], table.shape[1], None
    _need(positions, torch.int64, (tokens,), "positions", device)
    return table.shape[0], table.shape[1], positions.data_ptr()


def rotary_apply(x, table, positions=None, interleaved=False, backward=False, out=None, stream=None):
    """bf16 [T, heads, D]: the first rot channels of every head of x (whose
    tokens may lie apart: a slice of a fused projection) turned by the rows
    positions (int64 [T]; None: row t for token t) of table (fp32 [rows, rot],
    see rotary_table).  Pairs are channels i and i + rot / 2, or neighbours
    with interleaved.  backward: by the negative angles, the gradient.  Tokens
    with a negative position are copied.  out may be x."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be [T, heads, D]")
    device = _current(x, "x")
    t, heads, d = x.shape
    x_step = _need_heads(x, heads, d, "x", device)
    rows, rot, at = _rotary(table, positions, t, device)
    if out is None:
        out, out_step = _empty((t, heads, d), torch.bfloat16, x.device, stream), heads * d
    else:
        out_step = _need_heads(out, heads, d, "out", device)
        if out.shape[0] != t:
            raise ValueError("x and out disagree on T")
    st = lib().rotary_apply(x.data_ptr(), x_step, table.data_ptr(), rows, at, out.data_ptr(), out_step, t, heads, d, rot,
                            bool(interleaved), bool(backward), _stream(stream))
    if st != I8QL_OK:
        _check(st, "rotary_apply")
    return out


def kv_cache_store_rotary(q, k, v, table, slots, codes, params, positions=None, interleaved=False, q_out=None,
                          stream=None):
    """rotary_apply on q and k and kv_cache_store of the turned keys and v in one
    launch.  Returns the turned queries, bf16 [T, q_heads, head_dim] (q_out may
    be q; None with q = None, which stores alone)."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be [T, heads, head_dim]")
    t, _, d = k.shape
    pages, heads, page, bits, device = _kv_cache(codes, params, d)
    k_step = _need_heads(k, heads, d, "k", device)
    v_step = _need_heads(v, heads, d, "v", device)
    if v.shape[0] != t:
        raise ValueError("k and v disagree on T")
    _need(slots, torch.int64, (t,), "slots", device)
    rows, rot, at = _rotary(table, positions, t, device)
    hq = q_step = q_out_step = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [T, q_heads, head_dim]")
        hq = q.shape[1]
        q_step = _need_heads(q, hq, d, "q", device)
        if q.shape[0] != t:
            raise ValueError("q and k disagree on T")
        if q_out is None:
            q_out, q_out_step = _empty((t, hq, d), torch.bfloat16, codes.device, stream), hq * d
        else:
            q_out_step = _need_heads(q_out, hq, d, "q_out", device)
            if q_out.shape[0] != t:
                raise ValueError("q and q_out disagree on T")
    elif q_out is not None:
        raise ValueError("q_out without q")
    st = lib().kv_cache_store_rotary(_ptr(q), q_step, _ptr(q_out), q_out_step, k.data_ptr(), v.data_ptr(), k_step, v_step,
                                     table.data_ptr(), rows, at, slots.data_ptr(), codes.data_ptr(), params.data_ptr(),
                                     t, hq, heads, d, bits, page, pages, rot, bool(interleaved), _stream(stream))
    if st != I8QL_OK:
        _check(st, "kv_cache_store_rotary")
    return q_out


# ---------------------------------------------------------------- eviction from the key/value cache

def i8ql_kv_weights_workspace(batch, tokens, q_heads, heads, head_dim, bits, page_size, table_width, max_q=1) -> int:
    """Bytes of workspace a kv_cache_weights call of these sizes takes on the
    current device."""
    n = ctypes.c_int64(0)
    _check(lib().i8ql_kv_weights_workspace(batch, tokens, q_heads, heads, head_dim, bits, page_size, table_width, max_q,
                                           ctypes.byref(n)), "i8ql_kv_weights_workspace")
    return n.value


@functools.lru_cache(maxsize=1024)
def _weights_workspace_size(device: int, *sizes) -> int:
    """The same, asked once per device and sizes (a function of those alone)."""
    return i8ql_kv_weights_workspace(*sizes)


def kv_cache_weights(q, codes, params, page_table, kv_lens, weights, q_offsets=None, max_q=None, window=0, scale=None,
                     previous=None, workspace=None, stream=None):
    """Attention weights summed per cached token and head: weights (fp32
    [num_pages, heads, page_size]) = previous (the same; may be weights; None:
    nothing yet) of the tokens cached before this call's queries, plus the
    softmax weights of the query rows that see a token.  The other arguments as
    kv_cache_attention's, max_q being the most query tokens a sequence has (with
    q_offsets and without max_q all are taken for one sequence's: a batch of
    single tokens should say 1).
    Tokens that no query sees keep their weights.  Returns weights."""
    if q.dim() != 3:
        raise ValueError("q must be [T, q_heads, head_dim]")
    t, hq, d = q.shape
    pages, heads, page, bits, device = _kv_cache(codes, params, d)
    q_step = _need_heads(q, hq, d, "q", device)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, width]")
    b, width = page_table.shape
    _need(page_table, torch.int32, (b, width), "page_table", device)
    _need(kv_lens, torch.int32, (b,), "kv_lens", device)
    _need(weights, torch.float32, (pages, heads, page), "weights", device)
    if previous is not None:
        _need(previous, torch.float32, (pages, heads, page), "previous", device)
    if q_offsets is not None:
        _need(q_offsets, torch.int32, (b + 1,), "q_offsets", device)
    if max_q is None:
        max_q = 1 if q_offsets is None else t
    max_q = min(max_q, t)
    if workspace is None:
        size = 0
        if t and b:
            size = _weights_workspace_size(torch.cuda.current_device(), b, t, hq, heads, d, bits, page, width, max_q)
        if size:
            workspace = _empty((size,), torch.uint8, codes.device, stream)
    else:
        _need(workspace, torch.uint8, (workspace.numel(),), "workspace", device)
        size = workspace.numel()
    st = lib().kv_cache_weights(q.data_ptr(), q_step, codes.data_ptr(), params.data_ptr(), page_table.data_ptr(), width,
                                kv_lens.data_ptr(), None if q_offsets is None else q_offsets.data_ptr(),
                                None if previous is None else previous.data_ptr(), weights.data_ptr(), b, t, hq, heads,
                                d, bits, page, pages, max_q, window, d ** -0.5 if scale is None else scale,
                                None if workspace is None else workspace.data_ptr(), size, _stream(stream))
    if st != I8QL_OK:
        _check(st, "kv_cache_weights")
    return weights


def kv_cache_evict(codes, params, weights, page_table, kv_lens, budget, first=0, last=0, new_table=None, new_lens=None,
                   kept=None, stream=None):
    """Cuts every sequence to at most `budget` tokens: per head its first
    `first` and last `last` tokens stay, and those between with the largest
    weights (fp32 [num_pages, heads, page_size], see kv_cache_weights); codes,
    params and weights move to the front of the sequence's pages, or to those
    of new_table (int32 [B, width], pages that no sequence of the call
    occupies).  Returns (new_lens int32 [B], kept int32 [B, heads, budget]: the
    kept tokens' indices, -1 behind the last)."""
    if codes.dim() != 5:
        raise ValueError("codes must be [num_pages, 2, heads, page_size, head_dim * bits / 8]")
    row = codes.shape[4]  # (only the bytes of a row count here)
    d, bits = {32: (64, 4), 64: (128, 4), 128: (128, 8)}.get(row, (row, 8))
    pages, heads, page, bits, device = _kv_cache(codes, params, d)
    _need(weights, torch.float32, (pages, heads, page), "weights", device)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, width]")
    b, width = page_table.shape
    _need(page_table, torch.int32, (b, width), "page_table", device)
    _need(kv_lens, torch.int32, (b,), "kv_lens", device)
    new_width = width
    if new_table is not None:
        if new_table.dim() != 2:
            raise ValueError("new_table must be [B, width]")
        new_width = new_table.shape[1]
        _need(new_table, torch.int32, (b, new_width), "new_table", device)
    if budget < 1:
        raise ValueError("budget must be at least 1")
    if new_lens is None:
        new_lens = _empty((b,), torch.int32, codes.device, stream)
    else:
        _need(new_lens, torch.int32, (b,), "new_lens", device)
    if kept is None:
        kept = _empty((b, heads, budget), torch.int32, codes.device, stream)
    else:
        _need(kept, torch.int32, (b, heads, budget), "kept", device)
    st = lib().kv_cache_evict(codes.data_ptr(), params.data_ptr(), weights.data_ptr(), page_table.data_ptr(), width,
                              kv_lens.data_ptr(), None if new_table is None else new_table.data_ptr(), new_width,
                              new_lens.data_ptr(), kept.data_ptr(), b, heads, d, bits, page, pages, budget, first, last,
                              _stream(stream))
    if st != I8QL_OK:
        _check(st, "kv_cache_evict")
    return new_lens, kept
