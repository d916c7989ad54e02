"""Thin Python binding of libkaio_qkv (C ABI in include/kaio_qkv.h).

Argument marshalling only: shape/dtype checks on the torch tensors, output
allocation with torch, and one ctypes call per operation. Every step of the
computation runs in the library's CUDA kernels; there is no CPU path. If the
library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import operator
import os
import re
import struct
from typing import Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkaio_qkv.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "kaio_qkv.h")

KAIO_OK = 0
KAIO_ERR_INVALID_VALUE = 1
KAIO_ERR_MISALIGNED = 2
KAIO_ERR_UNSUPPORTED_DEVICE = 3
KAIO_ERR_CUDA = 4
KAIO_ERR_DEVICE_TIMEOUT = 5

KAIO_PAGED_ATTENTION_COUNTERS = 4096

KAIO_DTYPE_F32, KAIO_DTYPE_F64, KAIO_DTYPE_F16, KAIO_DTYPE_BF16, KAIO_DTYPE_S8, KAIO_DTYPE_U8 = range(6)

_lib = None

_vp, _u32, _i32 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int
_SIGNATURES = {
    "kaio_qkv_project_int4": ([_vp] * 10 + [_u32, _u32, _u32, _vp], _i32),
    "kaio_qkv_project_int4_noalloc": ([_vp] * 10 + [_u32, _u32, _u32, _vp], _i32),
    "kaio_debug_decode_wait_limit": ([_vp] * 10 + [_u32, _u32, _u32, ctypes.c_uint64, _vp], _i32),
    "kaio_matmul_tc": ([_vp, _vp, _vp, _u32, _u32, _u32, _vp], _i32),
    "kaio_matmul_tc_backward": ([_vp] * 5 + [_u32, _u32, _u32, _vp], _i32),
    "kaio_matmul_tc_f16": ([_vp, _vp, _vp, _u32, _u32, _u32, _vp], _i32),
    "kaio_matmul_tc_backward_f16": ([_vp] * 5 + [_u32, _u32, _u32, _vp], _i32),
    "kaio_dequant_int4_debug": ([_vp, _vp, _vp, _u32, _u32, _i32, _vp], _i32),
    "kaio_dequantize_per_group_backward": ([_i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp], _i32),
    "kaio_dequantize_per_group": ([_i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp], _i32),
    "kaio_qkv_project_int8": ([_vp] * 4 + [ctypes.c_float] * 3 + [_vp] * 3 + [_u32, _u32, _u32, _vp], _i32),
    "kaio_rope": ([_vp, _vp], _i32),
    "kaio_rope_append": ([_vp, _vp], _i32),
    "kaio_paged_attention": ([_vp, _vp], _i32),
    "kaio_paged_attention_scored": ([_vp, _vp], _i32),
    "kaio_debug_paged_attention_wait_limit": ([_vp, ctypes.c_uint64, _vp], _i32),
    "kaio_paged_attention_workspace": ([_vp], _i32),
    "kaio_cache_copy_pages": ([_vp, _vp], _i32),
    "kaio_cache_fork": ([_vp, _vp], _i32),
    "kaio_cache_append": ([_vp, _vp], _i32),
    "kaio_cache_truncate": ([_vp, _vp], _i32),
    "kaio_cache_compact": ([_vp, _vp], _i32),
    "kaio_debug_cache_cluster_limit": ([_i32, _vp, _i32, _vp], _i32),
    "kaio_qkv_path": ([_u32], _i32),
    "kaio_last_error": ([], ctypes.c_char_p),
    "kaio_device_status": ([], _i32),
    "kaio_status_string": ([_i32], ctypes.c_char_p),
}


# Argument blocks of the entries that take one (the structs of include/kaio_qkv.h,
# field by field), filled by one pack() each.
_ROPE_ARGS = struct.Struct("@I7i4i4i9P15q")
_PAGED_ARGS = struct.Struct("@I13ifi9PQ11q")
_PAGED_SCORED_ARGS = struct.Struct("@I13ifi9PQ11qfi3P")
_CACHE_COPY_ARGS = struct.Struct("@I7i4P")
_CACHE_ARGS = struct.Struct("@I7iq9P")


class KaioError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_string(status)}: {message}")
        self.status = status


def lib():
    """Load the shared library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def header_functions():
    """Names of the functions declared in include/kaio_qkv.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:int|const char\*)\s+(kaio_\w+)\s*\(", text, re.M)))


def status_string(status: int) -> str:
    try:
        return lib().kaio_status_string(status).decode()
    except Exception:  # pragma: no cover - library missing
        return f"status {status}"


def last_error() -> str:
    return lib().kaio_last_error().decode()


def check(status: int) -> None:
    if status != KAIO_OK:
        raise KaioError(status, last_error())


# ------------------------------------------------------------------ helpers
def _torch():
    import torch
    return torch


def _stream_ptr(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _need(t, name, dtypes, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device (no CPU fallback)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major, no strides of its own)")
    if t.dim() != 2:
        raise ValueError(f"{name} must be rank 2, got shape {tuple(t.shape)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.requires_grad:
        raise ValueError(f"{name} has gradient tracking enabled; these ops are forward-only: detach() it")


_PACKED = None


def _packed_dtypes():
    global _PACKED
    if _PACKED is None:
        torch = _torch()
        _PACKED = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
    return _PACKED


# ------------------------------------------------------------------ public API
def qkv_project_int4(x, w_q_packed, w_k_packed, w_v_packed, scales_q, scales_k, scales_v,
                     out: Optional[Tuple] = None, stream=None):
    """Fused W4A16 QKV projection: returns (q, k, v), each f16 [M, N].

    x f16 [M, K]; w_*_packed int32/uint32 [K/8, N] (8 signed INT4 per word, nibble
    i = K-row 8r+i); scales_* f16 [K/128, N].
    """
    torch = _torch()
    _need(x, "x", (torch.float16,))
    m, k = x.shape
    if k % 128:
        raise ValueError(f"K ({k}) must be a multiple of group_size (128)")
    n = w_q_packed.shape[1] if w_q_packed.dim() == 2 else -1
    for name, t in (("w_q_packed", w_q_packed), ("w_k_packed", w_k_packed), ("w_v_packed", w_v_packed)):
        _need(t, name, _packed_dtypes(), (k // 8, n))
    for name, t in (("scales_q", scales_q), ("scales_k", scales_k), ("scales_v", scales_v)):
        _need(t, name, (torch.float16,), (k // 128, n))
    if out is None:
        out = tuple(torch.empty((m, n), dtype=torch.float16, device=x.device) for _ in range(3))
    for name, t in zip("qkv", out):
        _need(t, name, (torch.float16,), (m, n))
    check(lib().kaio_qkv_project_int4(
        x.data_ptr(), w_q_packed.data_ptr(), w_k_packed.data_ptr(), w_v_packed.data_ptr(),
        scales_q.data_ptr(), scales_k.data_ptr(), scales_v.data_ptr(),
        out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), m, n, k, _stream_ptr(stream)))
    return out


def qkv_project_int8(x, w_q_packed, w_k_packed, w_v_packed, scale_q: float, scale_k: float,
                     scale_v: float, out: Optional[Tuple] = None, stream=None):
    """Fused W8A16 QKV projection: returns (q, k, v), each f16 [M, N].

    x f16 [M, K]; w_*_packed int32/uint32 [K/4, N] (4 signed INT8 per word,
    byte i = K-row 4r+i); scale_* one float per projection (passed as f32).
    """
    torch = _torch()
    _need(x, "x", (torch.float16,))
    m, k = x.shape
    if k % 128:
        raise ValueError(f"K ({k}) must be a multiple of 128")
    n = w_q_packed.shape[1] if w_q_packed.dim() == 2 else -1
    for name, t in (("w_q_packed", w_q_packed), ("w_k_packed", w_k_packed), ("w_v_packed", w_v_packed)):
        _need(t, name, _packed_dtypes(), (k // 4, n))
    if out is None:
        out = tuple(torch.empty((m, n), dtype=torch.float16, device=x.device) for _ in range(3))
    for name, t in zip("qkv", out):
        _need(t, name, (torch.float16,), (m, n))
    check(lib().kaio_qkv_project_int8(
        x.data_ptr(), w_q_packed.data_ptr(), w_k_packed.data_ptr(), w_v_packed.data_ptr(),
        float(scale_q), float(scale_k), float(scale_v),
        out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), m, n, k, _stream_ptr(stream)))
    return out


def matmul_tc(a, b, out=None, stream=None, out_dtype=None):
    """C = A @ B on the tensor cores: a f16 [M, K], b f16 [K, N] -> [M, N] in
    f32 (default) or f16 (rounded in the kernel's epilogue)."""
    torch = _torch()
    _need(a, "a", (torch.float16,))
    _need(b, "b", (torch.float16,))
    m, k = a.shape
    k2, n = b.shape
    if k != k2:
        raise ValueError(f"K mismatch between inputs: a is [{m}, {k}], b is [{k2}, {n}]")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32
    if out_dtype not in (torch.float32, torch.float16):
        raise ValueError(f"out_dtype must be float32 or float16, got {out_dtype}")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=a.device)
    _need(out, "c", (out_dtype,), (m, n))
    fn = lib().kaio_matmul_tc if out_dtype == torch.float32 else lib().kaio_matmul_tc_f16
    check(fn(a.data_ptr(), b.data_ptr(), out.data_ptr(), m, n, k, _stream_ptr(stream)))
    return out


def matmul_tc_backward(a, b, g, stream=None, out_dtype=None, out=None):
    """(dA, dB) = (G @ B^T, A^T @ G) for C = A @ B, with g f16 [M, N]; the
    results are f32 (default) or f16 (rounded in the kernels' epilogues),
    written into ``out = (da, db)`` when given."""
    torch = _torch()
    _need(a, "a", (torch.float16,))
    _need(b, "b", (torch.float16,))
    m, k = a.shape
    n = b.shape[1]
    _need(b, "b", (torch.float16,), (k, n))
    _need(g, "g", (torch.float16,), (m, n))
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if out_dtype not in (torch.float32, torch.float16):
        raise ValueError(f"out_dtype must be float32 or float16, got {out_dtype}")
    if out is None:
        da = torch.empty((m, k), dtype=out_dtype, device=a.device)
        db = torch.empty((k, n), dtype=out_dtype, device=a.device)
    else:
        da, db = out
        _need(da, "da", (out_dtype,), (m, k))
        _need(db, "db", (out_dtype,), (k, n))
    fn = lib().kaio_matmul_tc_backward if out_dtype == torch.float32 else lib().kaio_matmul_tc_backward_f16
    check(fn(a.data_ptr(), b.data_ptr(), g.data_ptr(), da.data_ptr(), db.data_ptr(), m, n, k,
             _stream_ptr(stream)))
    return da, db


def dequant_int4_debug(w_packed, scales, variant: int = 0, stream=None):
    """f16 [K, N] dequantised weights, exactly as the kernels build them."""
    torch = _torch()
    _need(w_packed, "w", _packed_dtypes())
    rows, n = w_packed.shape
    k = rows * 8
    _need(scales, "s", (torch.float16,), (k // 128, n))
    out = torch.empty((k, n), dtype=torch.float16, device=w_packed.device)
    check(lib().kaio_dequant_int4_debug(w_packed.data_ptr(), scales.data_ptr(), out.data_ptr(),
                                        k, n, variant, _stream_ptr(stream)))
    return out


def qkv_path(m: int) -> int:
    return lib().kaio_qkv_path(m)


def device_status() -> None:
    """Synchronise and raise if a kernel reported a bounded-wait timeout."""
    check(lib().kaio_device_status())


def _float_code(dtype):
    torch = _torch()
    codes = {torch.float32: KAIO_DTYPE_F32, torch.float64: KAIO_DTYPE_F64,
             torch.float16: KAIO_DTYPE_F16, torch.bfloat16: KAIO_DTYPE_BF16}
    if dtype not in codes:
        raise TypeError(f"dtype {dtype} is not one of float32, float64, float16, bfloat16")
    return codes[dtype]


def dequantize_per_group_backward(dy, scale, group: int, q_dtype=None, out=None, stream=None):
    """dx[i, j] = dy[i, j] * scale[i, j // group] (straight-through backward of
    the per-group dequantisation), for dy [outer, axis] and scale
    [outer, axis // group] of one float type. q_dtype (int8 or uint8, default
    int8) is the forward's quantised type; out may be dy itself (in place)."""
    torch = _torch()
    fdt = (torch.float32, torch.float64, torch.float16, torch.bfloat16)
    _need(dy, "dy", fdt)
    outer, axis = dy.shape
    if group <= 0 or axis % group != 0:
        raise ValueError(f"group ({group}) must be > 0 and divide axis ({axis})")
    _need(scale, "scale", (dy.dtype,), (outer, axis // group))
    q_dtype = torch.int8 if q_dtype is None else q_dtype
    qcode = {torch.int8: KAIO_DTYPE_S8, torch.uint8: KAIO_DTYPE_U8}.get(q_dtype)
    if qcode is None:
        raise TypeError("q_dtype must be torch.int8 or torch.uint8")
    if out is None:
        out = torch.empty_like(dy)
    _need(out, "dx", (dy.dtype,), (outer, axis))
    check(lib().kaio_dequantize_per_group_backward(_float_code(dy.dtype), qcode, outer, axis, group,
                                                   dy.data_ptr(), scale.data_ptr(), out.data_ptr(),
                                                   _stream_ptr(stream)))
    return out


def dequantize_per_group(q, scale, group: int, out=None, stream=None):
    """out[i, j] = T(q[i, j]) * scale[i, j // group] for q int8 or uint8
    [outer, axis] and scale [outer, axis // group] of float type T."""
    torch = _torch()
    _need(q, "q", (torch.int8, torch.uint8))
    outer, axis = q.shape
    if group <= 0 or axis % group != 0:
        raise ValueError(f"group ({group}) must be > 0 and divide axis ({axis})")
    _need(scale, "scale", (torch.float32, torch.float64, torch.float16, torch.bfloat16), (outer, axis // group))
    if out is None:
        out = torch.empty((outer, axis), dtype=scale.dtype, device=q.device)
    _need(out, "out", (scale.dtype,), (outer, axis))
    qcode = KAIO_DTYPE_S8 if q.dtype == torch.int8 else KAIO_DTYPE_U8
    check(lib().kaio_dequantize_per_group(qcode, _float_code(scale.dtype), outer, axis, group,
                                          q.data_ptr(), scale.data_ptr(), out.data_ptr(), _stream_ptr(stream)))
    return out


# ------------------------------------------- rotary positions, paged attention
# These run once per layer and step, on a few microseconds of GPU work when there
# are few tokens, so their checks are written to be cheap: one expression for a
# tensor that is as it should be (_fits), and _refuse to say what is wrong with
# one that is not.
_f16_codes = None


def _f16_code(dtype, name):
    global _f16_codes
    if _f16_codes is None:
        torch = _torch()
        _f16_codes = {torch.float16: KAIO_DTYPE_F16, torch.bfloat16: KAIO_DTYPE_BF16}
    code = _f16_codes.get(dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {dtype}, expected torch.float16 or torch.bfloat16")
    return code


def _refuse(t, name, dtype, shape):
    """Raises what is wrong with a tensor that may have strides of its own (a dense
    last dimension); None in ``shape`` takes any size."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU fallback)")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    got = t.shape
    if len(got) != len(shape):
        raise ValueError(f"{name} must be rank {len(shape)}, got shape {tuple(got)}")
    for g, want in zip(got, shape):
        if want is not None and g != want:
            raise ValueError(f"{name} has shape {tuple(got)}, expected {tuple(shape)}")
    if t.requires_grad:
        raise ValueError(f"{name} has gradient tracking enabled; these ops are forward-only: detach() it")
    raise ValueError(f"{name} must have a dense last dimension (strides {t.stride()})")


def _strides(t, name, dtype, shape):
    """Strides of a tensor of exactly this type and shape, on a GPU, without
    gradient tracking and with a dense last dimension; anything else raises."""
    try:
        strides = t.stride()
        if (t.dtype is dtype and t.shape == shape and t.is_cuda and not t.requires_grad
                and (strides[-1] == 1 or shape[-1] <= 1)):
            return strides
    except (AttributeError, TypeError):
        pass
    _refuse(t, name, dtype, shape)


def _size(t, name, dtype, rank, dim):
    """One size of a tensor whose other sizes _strides checks afterwards."""
    try:
        return t.shape[dim]
    except (AttributeError, IndexError, TypeError):
        _refuse(t, name, dtype, (None,) * rank)


def _rank3(x, name):
    """(type code, dtype, shape) of an activation tensor [tokens, heads, columns]."""
    try:
        dtype, shape = x.dtype, x.shape
        if len(shape) == 3:
            return _f16_code(dtype, name), dtype, shape
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    raise ValueError(f"{name} must be rank 3, got shape {tuple(shape)}")


def _raw_stream(t, stream) -> int:
    """The stream to run on: the one given, or the current one of t's device."""
    if stream is not None:
        return int(stream.cuda_stream)
    return _current_raw_stream(t.get_device())


def _int32(v, name):
    try:
        i = operator.index(v)
    except TypeError:
        raise TypeError(f"{name} must be an integer, got {type(v).__name__}") from None
    if not -2 ** 31 <= i < 2 ** 31:
        raise ValueError(f"{name} ({i}) is out of range")
    return i


def _pack(fields, *values):
    """An argument block; sizes of tensors that its fields do not hold raise."""
    try:
        return fields.pack(*values)
    except struct.error as e:
        raise ValueError(f"a tensor's size is out of range ({e})") from None


def _torch_stream(stream, device):
    """The stream given as torch's own (None: the current one, for torch.cuda.stream)."""
    torch = _torch()
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream.cuda_stream), device=device)


def _empty(shape, dtype, device, stream):
    """A new result. It belongs to the stream that the kernel runs on: on another one's
    memory that stream's earlier work might not be done, and its later work would get the
    memory back while the kernel still writes."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _current_raw_stream(device: int) -> int:
    global _current_raw_stream
    torch = _torch()
    # The same value as torch.cuda.current_stream().cuda_stream, without making a
    # Stream object (3 of the 4 microseconds that a call may take on the host).
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: int(torch.cuda.current_stream(d).cuda_stream))
    return _current_raw_stream(device)


def _rope_axes(positions, tokens, sections, pairs):
    """(axes, axis stride, sections padded to four) of a positions tensor [T] or [axes, T]."""
    int32 = _torch().int32
    if getattr(positions, "ndim", None) == 1:
        _strides(positions, "positions", int32, (tokens,))
        axes, stride = 1, 0
    else:
        axes = _size(positions, "positions", int32, 2, 0)
        stride = _strides(positions, "positions", int32, (axes, tokens))[0]
    if sections is None:
        if axes != 1:
            raise ValueError(f"positions has {axes} axes: sections has to say how many pairs each one turns")
        return 1, stride, (pairs, 0, 0, 0)
    if len(sections) != axes or axes > 4:
        raise ValueError(f"sections {tuple(sections)} does not fit positions with {axes} axes (1 to 4)")
    return axes, stride, (*(_int32(s, "sections") for s in sections), 0, 0, 0)[:4]


_host_module = None


def _host():
    """The module that makes an ordinary call in one step (csrc/host_calls.cpp): its
    functions return the result, or None to leave a call to the code here. False
    where it was not built."""
    global _host_module
    if _host_module is None:
        L = lib()
        _torch()                                           # its libraries have to be loaded first
        try:
            from . import _host as module
        except ImportError:
            _host_module = False
        else:
            module.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                          for f in (L.kaio_rope, L.kaio_rope_append, L.kaio_paged_attention)))
            module.bind_more(*(ctypes.cast(f, ctypes.c_void_p).value
                               for f in (L.kaio_paged_attention_scored, L.kaio_cache_copy_pages, L.kaio_cache_fork,
                                         L.kaio_cache_append, L.kaio_cache_truncate, L.kaio_cache_compact)))
            _host_module = module
    return _host_module


def rope(x, positions, inv_freq, sections=None, interleaved: bool = False, inverse: bool = False, out=None,
         stream=None):
    """Rotary positions: returns x [T, H, D] (f16 or bf16) with its first 2 * R
    columns turned by positions[a(i), t] * inv_freq[i], pair by pair.

    positions int32 [T] or [axes, T]; inv_freq f32 [R]; sections: how many
    consecutive pairs each axis turns (default: all by the one axis). Pairs are
    columns (i, i + R), or (2i, 2i + 1) if interleaved. inverse turns the other
    way: the gradient of the rotation with respect to x, given that of its
    result. out may be x itself. A new result belongs to ``stream`` (default: the
    current one).
    """
    host = _host_module or _host()
    if host:
        done = host.rope(x, positions, inv_freq, sections, interleaved, inverse, out, stream)
        if done is not None:
            return done
    torch = _torch()
    code, dtype, shape = _rank3(x, "x")
    t, h, d = shape
    xs = _strides(x, "x", dtype, shape)
    pairs = _size(inv_freq, "inv_freq", torch.float32, 1, 0)
    _strides(inv_freq, "inv_freq", torch.float32, (pairs,))
    axes, axis_stride, sec = _rope_axes(positions, t, sections, pairs)
    if out is None:
        out = _empty(shape, dtype, x.device, stream)
        os_ = (h * d, d)
    else:
        os_ = _strides(out, "out", dtype, shape)
    args = _pack(_ROPE_ARGS, _ROPE_ARGS.size, code, t, h, 0, d, pairs, axes, *sec,
                 bool(interleaved), bool(inverse), 0, 0,
                 x.data_ptr(), 0, 0, out.data_ptr(), 0, 0, positions.data_ptr(), inv_freq.data_ptr(), 0,
                 xs[0], xs[1], os_[0], os_[1], 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, axis_stride)
    check(lib().kaio_rope(args, _raw_stream(x, stream)))
    return out


def rope_append(q, k, v, positions, inv_freq, k_cache, v_cache, slots, sections=None, interleaved: bool = False,
                q_out=None, stream=None):
    """Rotates q and k as ``rope`` does and writes the rotated k and the unchanged
    v into a paged cache, in one launch. Returns the rotated q.

    q [T, H, D], k and v [T, KH, D]; k_cache and v_cache [pages, page_size, KH, D]
    (any strides with a dense last dimension, such as a transposed [pages, KH,
    page_size, D]); slots int32 [T]: page * page_size + place in the page for each
    token, or -1 to store nothing. q_out may be q itself; k and v may then lie beside
    it in one packed buffer. A new result belongs to ``stream``, as for ``rope``.
    """
    host = _host_module or _host()
    if host:
        done = host.rope_append(q, k, v, positions, inv_freq, k_cache, v_cache, slots, sections, interleaved, q_out,
                                stream)
        if done is not None:
            return done
    torch = _torch()
    code, dtype, shape = _rank3(q, "q")
    t, h, d = shape
    qs = _strides(q, "q", dtype, shape)
    kh = _size(k, "k", dtype, 3, 1)
    ks = _strides(k, "k", dtype, (t, kh, d))
    vs = _strides(v, "v", dtype, (t, kh, d))
    pages, page_size = _size(k_cache, "k_cache", dtype, 4, 0), _size(k_cache, "k_cache", dtype, 4, 1)
    cache = (pages, page_size, kh, d)
    kc = _strides(k_cache, "k_cache", dtype, cache)
    vc = _strides(v_cache, "v_cache", dtype, cache)
    pairs = _size(inv_freq, "inv_freq", torch.float32, 1, 0)
    _strides(inv_freq, "inv_freq", torch.float32, (pairs,))
    _strides(slots, "slots", torch.int32, (t,))
    axes, axis_stride, sec = _rope_axes(positions, t, sections, pairs)
    if q_out is None:
        q_out = _empty(shape, dtype, q.device, stream)
        os_ = (h * d, d)
    else:
        os_ = _strides(q_out, "q_out", dtype, shape)
    args = _pack(_ROPE_ARGS, _ROPE_ARGS.size, code, t, h, kh, d, pairs, axes, *sec,
                 bool(interleaved), 0, pages, page_size,
                 q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(),
                 v_cache.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), slots.data_ptr(),
                 qs[0], qs[1], os_[0], os_[1], ks[0], ks[1], vs[0], vs[1], kc[0], kc[1], kc[2],
                 vc[0], vc[1], vc[2], axis_stride)
    check(lib().kaio_rope_append(args, _raw_stream(q, stream)))
    return q_out


def paged_attention_workspace(device=None, stream=None):
    """A workspace for ``paged_attention`` on a device: allocate it once and keep
    it. What has to be zero in it is zeroed on ``stream`` (default: the current one).
    That and the calls that use it must be ordered (one stream, or events)."""
    torch = _torch()
    n = ctypes.c_uint64()
    with torch.cuda.device(device), torch.cuda.stream(_torch_stream(stream, device)):
        check(lib().kaio_paged_attention_workspace(ctypes.byref(n)))
        workspace = torch.empty(n.value, dtype=torch.uint8, device="cuda")
        workspace[:KAIO_PAGED_ATTENTION_COUNTERS].zero_()
        return workspace


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, q_starts=None, max_new: Optional[int] = None,
                    scale: Optional[float] = None, causal: bool = True, window: int = 0, sinks: int = 0,
                    workspace=None, out=None, return_lse: bool = False, lse=None, stream=None, softcap: float = 0.0,
                    slopes=None, prefix_lens=None, doc_starts=None):
    """Attention of new tokens over a paged cache that already holds their keys
    and values. Returns out [T, H, D], or (out, lse f32 [T, H]) with return_lse.

    q [T, H, D] (f16 or bf16): the new tokens of all sequences, those of sequence
    b at q_starts[b]:q_starts[b + 1] (int32 [B + 1]; default: one token each);
    they are the last ones of its kv_lens[b] (int32 [B]) positions. k_cache and
    v_cache [pages, page_size, KH, D], any strides with a dense last dimension,
    page_size a power of two from 16 to 1024, H a multiple of KH; page_table
    int32 [B, P]. max_new: at least the largest number of new tokens of one
    sequence (default: T, or 1 without q_starts); it chooses the kernel, so give 1 for
    a batch of single tokens with q_starts. scale defaults to D ** -0.5.
    causal: a token sees positions up to its own; window: only the last `window`
    of them, and the first `sinks` positions besides. prefix_lens (int32 [B]): so many
    first positions all new tokens of the sequence see, also those that stand before them.
    doc_starts (int32 [T], not decreasing within a sequence): a token sees nothing before
    its document's begin. softcap (up to 256; 0: none): scores s become
    softcap * tanh(s / softcap); slopes (f32 [H]): they then lose slopes[h] for each
    position between token and key. A token that sees nothing gets zeros and lse = -inf.
    workspace: from ``paged_attention_workspace``;
    without one the call makes its own. New results and that workspace belong to
    ``stream`` (default: the current one).
    """
    scored = not (softcap == 0 and slopes is None and prefix_lens is None and doc_starts is None)
    host = _host_module or _host()
    if host:
        if scored:
            done = host.paged_attention_scored(q, k_cache, v_cache, page_table, kv_lens, q_starts, max_new, scale, causal,
                                               window, sinks, workspace, out, return_lse, lse, stream, softcap, slopes,
                                               prefix_lens, doc_starts)
        else:
            done = host.paged_attention(q, k_cache, v_cache, page_table, kv_lens, q_starts, max_new, scale, causal, window,
                                        sinks, workspace, out, return_lse, lse, stream)
        if done is not None:
            return done
    cap = ctypes.c_float(softcap).value
    if cap == 0 and softcap != 0:
        raise ValueError(f"softcap ({softcap}) is zero in 32 bits: it must be 0 or in (0, 256]")
    torch = _torch()
    int32 = torch.int32
    code, dtype, shape = _rank3(q, "q")
    t, h, d = shape
    qs = _strides(q, "q", dtype, shape)
    cache = k_cache.shape if hasattr(k_cache, "shape") else ()
    if len(cache) != 4:
        _refuse(k_cache, "k_cache", dtype, (None, None, None, d))
    pages, page_size, kh, _ = cache
    kc = _strides(k_cache, "k_cache", dtype, (pages, page_size, kh, d))
    vc = _strides(v_cache, "v_cache", dtype, cache)
    b = _size(kv_lens, "kv_lens", int32, 1, 0)
    _strides(kv_lens, "kv_lens", int32, (b,))
    max_pages = _size(page_table, "page_table", int32, 2, 1)
    ts = _strides(page_table, "page_table", int32, (b, max_pages))
    starts = 0
    if q_starts is not None:
        _strides(q_starts, "q_starts", int32, (b + 1,))
        starts = q_starts.data_ptr()
    if workspace is None:
        # on the call's own stream: zeroed before the kernel, and freed to that stream's later work
        workspace = paged_attention_workspace(q.device, stream)
    elif not (getattr(workspace, "is_cuda", False) and workspace.dtype is torch.uint8 and workspace.is_contiguous()):
        raise ValueError("workspace must be a dense uint8 CUDA tensor from paged_attention_workspace()")
    if out is None:
        out = _empty(shape, dtype, q.device, stream)
        os_ = (h * d, d)
    else:
        os_ = _strides(out, "out", dtype, shape)
    lse_ptr = 0
    if lse is not None:
        if _strides(lse, "lse", torch.float32, (t, h))[0] != h and t > 1:
            raise ValueError("lse must be contiguous")
        lse_ptr = lse.data_ptr()
    elif return_lse:
        lse = _empty((t, h), torch.float32, q.device, stream)
        lse_ptr = lse.data_ptr()
    if max_new is None:
        max_new = t if starts else 1
    if scale is None:
        scale = max(d, 1) ** -0.5
    more = 0, 0, 0
    if scored:
        if slopes is not None:
            _strides(slopes, "slopes", torch.float32, (h,))
        if prefix_lens is not None:
            _strides(prefix_lens, "prefix_lens", int32, (b,))
        if doc_starts is not None:
            _strides(doc_starts, "doc_starts", int32, (t,))
        more = tuple(0 if m is None else m.data_ptr() for m in (slopes, prefix_lens, doc_starts))
    fields = _PAGED_SCORED_ARGS if scored else _PAGED_ARGS
    args = _pack(fields, fields.size, code, b, t, h, kh, d, page_size, pages, max_pages,
                 _int32(max_new, "max_new"), bool(causal), _int32(window, "window"), _int32(sinks, "sinks"),
                 ctypes.c_float(scale).value, 0,
                 q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                 kv_lens.data_ptr(), starts, out.data_ptr(), lse_ptr, workspace.data_ptr(),
                 workspace.numel(),
                 qs[0], qs[1], os_[0], os_[1], kc[0], kc[1], kc[2], vc[0], vc[1], vc[2], ts[0],
                 *((cap, 0, *more) if scored else ()))
    entry = lib().kaio_paged_attention_scored if scored else lib().kaio_paged_attention
    check(entry(args, _raw_stream(q, stream)))
    return (out, lse) if return_lse else out


def cache_copy_pages(caches, src, dst, stream=None):
    """Copies page src[i] to page dst[i] of every cache, in one launch for up to 64 of them.

    caches: tensors [pages, page_size, KH, D] of one type (f16 or bf16) and shape, any
    strides with a dense last dimension: K and V of all layers. src and dst int32 [N];
    pairs with a page outside the cache (-1) are left out; no dst may be another pair's
    src or dst.
    """
    host = _host_module or _host()
    if host and host.cache_copy_pages(caches, src, dst, stream):
        return
    torch = _torch()
    caches = list(caches)
    n = _size(src, "src", torch.int32, 1, 0)
    _strides(src, "src", torch.int32, (n,))
    _strides(dst, "dst", torch.int32, (n,))
    if not caches:
        return
    shape = getattr(caches[0], "shape", ())
    dtype = getattr(caches[0], "dtype", None)
    if len(shape) != 4:
        _refuse(caches[0], "caches[0]", dtype, (None,) * 4)
    _f16_code(dtype, "caches[0]")
    pages, page_size, kh, d = shape
    steps = [s for i, c in enumerate(caches) for s in _strides(c, f"caches[{i}]", dtype, shape)[:3]]
    at = (ctypes.c_void_p * len(caches))(*(c.data_ptr() for c in caches))
    strides = (ctypes.c_int64 * len(steps))(*steps)
    args = _pack(_CACHE_COPY_ARGS, _CACHE_COPY_ARGS.size, len(caches), pages, page_size, kh, d, n, 0,
                 ctypes.addressof(at), ctypes.addressof(strides), src.data_ptr(), dst.data_ptr())
    check(lib().kaio_cache_copy_pages(args, _raw_stream(src, stream)))


def _cache_call(entry, page_refs, page_table, kv_lens, page_size, stream, tokens=0, max_moves=0, parents=None,
                q_starts=None, new_lens=None, slots=None, src=None, dst=None):
    int32 = _torch().int32
    pages = _size(page_refs, "page_refs", int32, 1, 0)
    _strides(page_refs, "page_refs", int32, (pages,))
    batch = _size(kv_lens, "kv_lens", int32, 1, 0)
    _strides(kv_lens, "kv_lens", int32, (batch,))
    width = _size(page_table, "page_table", int32, 2, 1)
    step = _strides(page_table, "page_table", int32, (batch, width))[0]
    for name, t, n in (("parents", parents, batch), ("q_starts", q_starts, batch + 1), ("new_lens", new_lens, batch)):
        if t is not None:
            _strides(t, name, int32, (n,))
    args = _pack(_CACHE_ARGS, _CACHE_ARGS.size, batch, width, pages, _int32(page_size, "page_size"), tokens, max_moves, 0,
                 step, page_refs.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(),
                 *(0 if t is None else t.data_ptr() for t in (parents, q_starts, new_lens, slots, src, dst)))
    check(entry(args, _raw_stream(page_refs, stream)))


def cache_fork(page_refs, page_table, kv_lens, parents, page_size: int, stream=None):
    """Row b of the books becomes a copy of row parents[b] (int32 [B]), all rows at once; a
    parent outside the batch leaves its row as it is. Pages are shared, none is copied.

    The books of a paged cache, which this and the following functions change in place:
    page_refs int32 [pages] (how many places of the table hold each page; 0: free),
    page_table int32 [B, P] and kv_lens int32 [B]; row b holds its first
    ceil(kv_lens[b] / page_size) places.
    """
    host = _host_module or _host()
    if not (host and host.cache_fork(page_refs, page_table, kv_lens, parents, page_size, stream)):
        _cache_call(lib().kaio_cache_fork, page_refs, page_table, kv_lens, page_size, stream, parents=parents)


def cache_append(page_refs, page_table, kv_lens, q_starts, tokens: int, page_size: int, stream=None):
    """Gives row b of the books q_starts[b + 1] - q_starts[b] new positions (int32 [B + 1],
    from 0 to ``tokens``; None: one each), in pages that are the lowest free ones.
    Returns (slots, src, dst): slots int32 [tokens] for ``rope_append``, and the pages
    to copy with ``cache_copy_pages`` before anything is written: where a row's last page
    is held elsewhere too, it gets dst[b] instead of src[b] (int32 [B]; -1: none).

    A row that does not fit its places, or the pool behind the rows before it, takes nothing:
    its slots are -1 and its books stay. Nothing raises then, and what ``paged_attention`` gives for its tokens
    means nothing: know the room before, or read slots (or kv_lens) back and leave the row out. New
    results belong to ``stream`` (default: the current one).
    """
    host = _host_module or _host()
    if host:
        done = host.cache_append(page_refs, page_table, kv_lens, q_starts, tokens, page_size, stream)
        if done is not None:
            return done
    int32 = _torch().int32
    batch = _size(kv_lens, "kv_lens", int32, 1, 0)
    tokens = _int32(tokens, "tokens")
    device = getattr(kv_lens, "device", None)
    slots, src, dst = (_empty((max(n, 0),), int32, device, stream) for n in (tokens, batch, batch))
    _cache_call(lib().kaio_cache_append, page_refs, page_table, kv_lens, page_size, stream, tokens=tokens,
                q_starts=q_starts, slots=slots, src=src, dst=dst)
    return slots, src, dst


def cache_truncate(page_refs, page_table, kv_lens, new_lens, page_size: int, stream=None):
    """Cuts row b of the books to new_lens[b] positions (int32 [B]) where it has more, and
    gives back the pages behind them; 0 frees the row."""
    host = _host_module or _host()
    if not (host and host.cache_truncate(page_refs, page_table, kv_lens, new_lens, page_size, stream)):
        _cache_call(lib().kaio_cache_truncate, page_refs, page_table, kv_lens, page_size, stream, new_lens=new_lens)


def cache_compact(page_refs, page_table, kv_lens, page_size: int, max_moves: int, stream=None):
    """Moves the highest used pages to the lowest free ones, up to ``max_moves``: renumbers the
    books and returns (src, dst), int32 [max_moves] filled up with -1, to be copied with
    ``cache_copy_pages``. New results belong to ``stream`` (default: the current one)."""
    host = _host_module or _host()
    if host:
        done = host.cache_compact(page_refs, page_table, kv_lens, page_size, max_moves, stream)
        if done is not None:
            return done
    int32 = _torch().int32
    max_moves = _int32(max_moves, "max_moves")
    device = getattr(kv_lens, "device", None)
    src, dst = (_empty((max(max_moves, 0),), int32, device, stream) for _ in range(2))
    _cache_call(lib().kaio_cache_compact, page_refs, page_table, kv_lens, page_size, stream, max_moves=max_moves,
                src=src, dst=dst)
    return src, dst
