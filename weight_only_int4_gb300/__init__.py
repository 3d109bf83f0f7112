"""weight_only_int4_gb300 -- W4A16 group-quantized linear layer for GB300.

A thin ctypes binding over libw4a16.so (C ABI in include/w4a16.h). Every
function below only checks and marshals its arguments (torch tensors ->
device pointers, the current CUDA stream) and calls the entry point of the
same name; all arithmetic runs in the library's CUDA kernels. There is no
CPU fallback: if the library is missing or the device is not a GB300, calls
raise.

    y = x @ W,   W[k, n] = (q[k, n] - z[k // g, n]) * s[k // g, n]

Operands (all CUDA tensors, contiguous):
    x        [M, K]    torch.float16 or torch.bfloat16
    qweight  [K/8, N]  torch.int32, nibble j of word [w, n] = q[8w + j, n]
    scales   [K/g, N]  same dtype as x
    qzeros   [K/g, N/8] torch.int32 (zero-point of column n in word n // 8 at
             bits 4 * (n % 8)), or None for the symmetric layer (z = 8).
             Zero-points in the activation dtype are rejected, never
             reinterpreted (as "Keep W4A16 zero-points packed at 4 bits
             instead of expanding to 2 bytes" requires, section "Testing").
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from .accounting import expanded_zero_bytes, layer_bytes, layer_flops  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libw4a16.so")

STATUS_NAMES = [
    "W4A16_OK", "W4A16_ERR_NULL", "W4A16_ERR_SHAPE", "W4A16_ERR_DTYPE", "W4A16_ERR_ALIGN",
    "W4A16_ERR_UNSUPPORTED", "W4A16_ERR_DEVICE", "W4A16_ERR_WORKSPACE", "W4A16_ERR_CUDA",
    "W4A16_ERR_TIMEOUT",
]
OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_DEVICE, ERR_WORKSPACE, \
    ERR_CUDA, ERR_TIMEOUT = range(10)
F16, BF16, F32 = 0, 1, 2
OP_GEMV, OP_GEMM, OP_MXFP4_MATMUL = 0, 1, 2
GATE_CHANNEL, GATE_TOKEN, GATE_ELEMENT = 0, 1, 2

# Every symbol include/w4a16.h declares, with (restype, argtypes).
_VP, _I64, _SZ, _INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
_LAYER_ARGS = [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _I64, _INT, _VP, _SZ, _VP]
SIGNATURES = {
    "w4a16_pack": (_INT, [_VP, _VP, _I64, _I64, _INT, _VP]),
    "w4a16_unpack": (_INT, [_VP, _VP, _I64, _I64, _INT, _VP]),
    "w4a16_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64, _I64]),
    "w4a16_capture_id": (ctypes.c_uint64, [_VP]),
    "w4a16_gemv": (_INT, _LAYER_ARGS),
    "w4a16_gemm": (_INT, _LAYER_ARGS),
    "w4a16_gemv_noalloc": (_INT, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _I64, _INT, _VP]),
    "w4a16_device_status": (_INT, [_VP]),
    "w4a16_selftest_wait_timeout": (_INT, [_VP]),
    "w4a16_selftest_mxfp4_matmul_plan": (_INT, [_I64, _I64, _I64, _INT, ctypes.POINTER(_INT)]),
    "w4a16_selftest_int8_matmul_plan": (_INT, [_I64, _I64, _I64, _INT, ctypes.POINTER(_INT)]),
    "w4a16_dequant": (_INT, [_VP, _VP, _VP, _VP, _I64, _I64, _I64, _INT, _VP]),
    "w4a16_mxfp4_dequant": (_INT, [_VP, _VP, _VP, _I64, _I64, _VP]),
    "w4a16_mxfp4_gemv": (_INT, [_VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _SZ, _VP]),
    "w4a16_mxfp4_gemm": (_INT, [_VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _SZ, _VP]),
    "w4a16_mxfp4_quantize": (_INT, [_VP, _VP, _VP, _I64, _I64, _INT, _INT, _VP]),
    "w4a16_mxfp4_dequant_rows": (_INT, [_VP, _VP, _VP, _I64, _I64, _VP]),
    "w4a16_mxfp4_tile_scales": (_INT, [_VP, _VP, _I64, _I64, _VP]),
    "w4a16_mxfp4_matmul": (_INT, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _INT, _VP, _SZ, _VP]),
    "w4a16_mxfp4_moe": (_INT, [_VP] * 7 + [_I64] * 5 + [_INT, _VP, _SZ, _VP]),
    "w4a16_mxfp4_moe_workspace_bytes": (_SZ, [_I64] * 5),
    "w4a16_int8_quantize": (_INT, [_VP, _VP, _VP, _I64, _I64, _INT, _VP]),
    "w4a16_int8_dequant": (_INT, [_VP, _VP, _VP, _I64, _I64, _INT, _VP]),
    "w4a16_int8_matmul": (_INT, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _INT, _VP, _SZ, _VP]),
    "w4a16_int8_matmul_workspace_bytes": (_SZ, [_I64] * 3),
    "w4a16_block_norm": (_INT, [_VP, _INT, _VP, _VP, _VP, _INT, ctypes.c_float, _VP, _VP, ctypes.c_float, _VP, _VP,
                                _VP, _I64, _I64, _INT, _VP]),
    "w4a16_status_string": (ctypes.c_char_p, [_INT]),
    "w4a16_abi_version": (_INT, []),
}


class W4A16Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else f"status {status}"
        super().__init__(f"{fn} failed: {name}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libw4a16.so (built by weight_only_int4_gb300.build). Raises if missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libw4a16.so not found at {path}; build it with "
                           "`python -m weight_only_int4_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().w4a16_status_string(status).decode()


def abi_version() -> int:
    return load_library().w4a16_abi_version()


_torch_module = None
_raw_stream = None   # device -> handle of its current stream; the object torch.cuda.current_stream() builds costs 3 us
_current_device = None
_dtype_codes = {}


def _torch():
    global _torch_module, _raw_stream, _current_device
    if _torch_module is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _dtype_codes.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
        _torch_module = torch
    return _torch_module


def _stream_ptr(stream=None) -> int:
    """Raw handle of `stream`, or of the current stream of the current device."""
    if stream is not None:
        return int(stream.cuda_stream)
    if _raw_stream is None:
        return int(_torch().cuda.current_stream().cuda_stream)
    return _raw_stream(_current_device())


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise W4A16Error(fn, status)


def _act_code(dtype) -> int:
    torch = _torch()
    if dtype == torch.float16:
        return F16
    if dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"activations must be float16 or bfloat16, got {dtype}")


def _dtype_code(dtype) -> int:
    _torch()
    code = _dtype_codes.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float16, bfloat16 or float32, got {dtype}")
    return code


def _cuda_contig(name: str, t, current: Optional[int] = None) -> None:
    """The kernels run on the current device (`current`, where the caller knows it)
    and take raw pointers: every tensor has to be there, and dense."""
    where = t.get_device()
    if where < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if where != (_current_device() if current is None else current):
        raise ValueError(f"{name} is on cuda:{where}, the current device is cuda:{_current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(name: str, t, shape, dtype, device, stream=None):
    """`t`, checked, or a new tensor that belongs to `stream` (the current one unless given)."""
    torch = _torch()
    if t is None:
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    _cuda_contig(name, t)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t


def pack(codes, dim: int, out=None, stream=None):
    """Pack uint8 4-bit codes [R, C] eight to an int32 word along `dim` (0: rows, 1: cols)."""
    torch = _torch()
    _cuda_contig("codes", codes)
    if codes.dtype != torch.uint8 or codes.dim() != 2:
        raise TypeError("codes must be a 2-D torch.uint8 tensor")
    R, C = codes.shape
    shape = (R // 8, C) if dim == 0 else (R, C // 8)
    out = _out("out", out, shape, torch.int32, codes.device)
    _check("w4a16_pack", load_library().w4a16_pack(codes.data_ptr(), out.data_ptr(), R, C, dim,
                                                   _stream_ptr(stream)))
    return out


def unpack(words, dim: int, out=None, stream=None):
    """Inverse of pack: int32 words -> uint8 codes [R, C]."""
    torch = _torch()
    _cuda_contig("words", words)
    if words.dtype != torch.int32 or words.dim() != 2:
        raise TypeError("words must be a 2-D torch.int32 tensor")
    W0, W1 = words.shape
    R, C = (W0 * 8, W1) if dim == 0 else (W0, W1 * 8)
    out = _out("out", out, (R, C), torch.uint8, words.device)
    _check("w4a16_unpack", load_library().w4a16_unpack(words.data_ptr(), out.data_ptr(), R, C, dim,
                                                       _stream_ptr(stream)))
    return out


def workspace_bytes(op: int, M: int, N: int, K: int, g: int) -> int:
    """Device workspace the op needs on the current device (0 if none)."""
    return int(load_library().w4a16_workspace_bytes(op, M, N, K, g))


def new_workspace(nbytes: int, device=None):
    """A zero-filled uint8 device workspace. Calls leave it zeroed where it must
    start at zero, so one workspace serves any number of calls, as long as no
    two calls that use it run at the same time."""
    torch = _torch()
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8,
                       device=torch.device("cuda") if device is None else device)


_workspaces = {}
_retired = []

# Bytes of FP32 partial sums per SM with which an op's workspace begins, as include/w4a16.h lays it out; ticket words,
# the part that must start at zero, follow.
_PARTIALS_PER_SM = {OP_GEMV: 136 << 10, OP_GEMM: 128 << 10, OP_MXFP4_MATMUL: 128 << 10}
# What must start at zero at the beginning of the others': barrier words, ticket words.
_MOE_CONTROL_BYTES = 256
_CONTROL_BYTES = {"mxfp4_moe": _MOE_CONTROL_BYTES, "int8_matmul": 4096}


def _zero_range(op, nbytes: int, sms: int):
    """(first, last + 1) of the bytes of a workspace that must start at zero."""
    if op in _PARTIALS_PER_SM:
        first = _PARTIALS_PER_SM[op] * sms
        return (first if first < nbytes else 0), nbytes
    return 0, min(_CONTROL_BYTES[op], nbytes)


def _captured_workspace(nbytes: int, device, op, sms: int):
    """A workspace whose zero fill will run on every replay of a graph: it covers
    what must start at zero and no more (all 20 MB of a product's partial sums
    would cost each replay 6 us)."""
    torch = _torch()
    ws = torch.empty(int(nbytes), dtype=torch.uint8, device=device)
    first, last = _zero_range(op, int(nbytes), sms)
    ws[first:last].zero_()
    return ws


def _cached_workspace(nbytes: int, device, stream, op: int):
    """One growing workspace per (device, stream, op): calls on one stream never
    overlap, and the GEMV and the GEMM lay out their workspaces differently.

    The workspace is allocated and zero-filled on the stream the call runs on,
    so the zero fill is ordered before the kernel and the caching allocator
    ties the memory to that stream. While that stream is captured the fill
    becomes a node of the graph, so every capture has workspaces of its own:
    each graph carries the fill that its kernels rely on, whichever is replayed
    first, and graphs replayed at the same time do not meet in one. A workspace
    of a capture, or one outgrown by a larger shape, is kept alive (not freed)
    until release_workspaces(): a graph may still replay into it."""
    torch = _torch()
    dev = device.index if device.index is not None else torch.cuda.current_device()
    if stream is not None:
        handle = int(stream.cuda_stream)
    else:
        handle = int(torch.cuda.current_stream(dev).cuda_stream) if _raw_stream is None else _raw_stream(dev)
    capture = load_library().w4a16_capture_id(handle)
    key = (dev, handle, op, capture)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        s = torch.cuda.current_stream(dev) if stream is None else stream
        with torch.cuda.stream(s):
            if capture:
                sms = torch.cuda.get_device_properties(dev).multi_processor_count
                fresh = _captured_workspace(nbytes, device, op, sms)
            else:
                fresh = new_workspace(nbytes, device)
        if ws is not None:
            _retired.append(ws)
        _workspaces[key] = ws = fresh
    return ws


def _workspace_args(ws):
    """(address, bytes) of a workspace, or of none."""
    if ws is None:
        return 0, 0
    _cuda_contig("workspace", ws)
    return ws.data_ptr(), ws.numel() * ws.element_size()


def release_workspaces() -> None:
    """Free the workspaces the binding allocated for calls made without one (one
    per device, stream and op, one more for each capture of the stream, plus any
    outgrown by larger shapes). Call it only
    when no such call is in flight, and only after dropping every CUDA graph
    captured through such calls: a captured graph replays into the workspace
    address it saw at capture time. The next call allocates a fresh, zeroed
    workspace."""
    _workspaces.clear()
    _retired.clear()


def _layer(fn_name: str, x, qweight, scales, qzeros, group_size: int, out=None, workspace=None,
           stream=None):
    torch = _torch()
    for name, t in (("x", x), ("qweight", qweight), ("scales", scales)):
        _cuda_contig(name, t)
    if x.dim() != 2 or qweight.dim() != 2 or scales.dim() != 2:
        raise ValueError("x, qweight and scales must be 2-D")
    dt = _act_code(x.dtype)
    if scales.dtype != x.dtype:
        raise TypeError(f"scales dtype {scales.dtype} differs from x dtype {x.dtype}")
    if qweight.dtype != torch.int32:
        raise TypeError(f"qweight must be torch.int32, got {qweight.dtype}")
    M, K = x.shape
    N = qweight.shape[1]
    if qweight.shape[0] * 8 != K:
        raise ValueError(f"qweight rows {qweight.shape[0]} do not match K/8 = {K / 8}")
    if K % group_size or scales.shape != (K // group_size, N):
        raise ValueError(f"scales shape {tuple(scales.shape)} does not match (K/g, N)")
    zp = 0
    if qzeros is not None:
        _cuda_contig("qzeros", qzeros)
        if qzeros.dtype != torch.int32:
            raise TypeError(f"qzeros must be packed torch.int32 [K/g, N/8]; got {qzeros.dtype} "
                            "(zero-points in the activation dtype are rejected)")
        if qzeros.shape != (K // group_size, N // 8):
            raise ValueError(f"qzeros shape {tuple(qzeros.shape)} does not match (K/g, N/8)")
        zp = qzeros.data_ptr()
    out = _out("out", out, (M, N), x.dtype, x.device)
    lib = load_library()
    sp = _stream_ptr(stream)
    if workspace is None:
        op = OP_GEMV if fn_name == "w4a16_gemv" else OP_GEMM
        need = lib.w4a16_workspace_bytes(op, M, N, K, group_size)
        workspace = _cached_workspace(need, x.device, stream, op) if need else None
    ws_ptr, ws_bytes = _workspace_args(workspace)
    _check(fn_name, getattr(lib, fn_name)(x.data_ptr(), qweight.data_ptr(), scales.data_ptr(), zp,
                                          out.data_ptr(), M, N, K, group_size, dt, ws_ptr, ws_bytes, sp))
    return out


def gemv(x, qweight, scales, qzeros: Optional[object], group_size: int, out=None, workspace=None,
         stream=None):
    """Decode path (1 <= M <= 16). Returns y [M, N] in x's dtype."""
    return _layer("w4a16_gemv", x, qweight, scales, qzeros, group_size, out, workspace, stream)


def gemm(x, qweight, scales, qzeros: Optional[object], group_size: int, out=None, workspace=None,
         stream=None):
    """Prefill path (any M >= 1, tcgen05 tensor cores). Returns y [M, N] in x's dtype."""
    return _layer("w4a16_gemm", x, qweight, scales, qzeros, group_size, out, workspace, stream)


def dequant(qweight, scales, qzeros: Optional[object], group_size: int, out=None, stream=None):
    """Dense dequantised copy W[k, n] = RN((q - z) * s) in the scales' dtype, [K, N]."""
    torch = _torch()
    for name, t in (("qweight", qweight), ("scales", scales)):
        _cuda_contig(name, t)
    if qweight.dim() != 2 or scales.dim() != 2:
        raise ValueError("qweight and scales must be 2-D")
    if qweight.dtype != torch.int32:
        raise TypeError(f"qweight must be torch.int32, got {qweight.dtype}")
    dt = _act_code(scales.dtype)
    K, N = qweight.shape[0] * 8, qweight.shape[1]
    if K % group_size or scales.shape != (K // group_size, N):
        raise ValueError(f"scales shape {tuple(scales.shape)} does not match (K/g, N)")
    zp = 0
    if qzeros is not None:
        _cuda_contig("qzeros", qzeros)
        if qzeros.dtype != torch.int32:
            raise TypeError(f"qzeros must be packed torch.int32 [K/g, N/8]; got {qzeros.dtype} "
                            "(zero-points in the activation dtype are rejected)")
        if qzeros.shape != (K // group_size, N // 8):
            raise ValueError(f"qzeros shape {tuple(qzeros.shape)} does not match (K/g, N/8)")
        zp = qzeros.data_ptr()
    out = _out("out", out, (K, N), scales.dtype, scales.device)
    _check("w4a16_dequant", load_library().w4a16_dequant(qweight.data_ptr(), scales.data_ptr(), zp, out.data_ptr(),
                                                         N, K, group_size, dt, _stream_ptr(stream)))
    return out


def _mx_weights(qweight, escale):
    torch = _torch()
    for name, t in (("qweight", qweight), ("escale", escale)):
        _cuda_contig(name, t)
    if qweight.dim() != 2 or escale.dim() != 2:
        raise ValueError("qweight and escale must be 2-D")
    if qweight.dtype != torch.int32:
        raise TypeError(f"qweight must be torch.int32, got {qweight.dtype}")
    if escale.dtype != torch.uint8:
        raise TypeError(f"escale must be torch.uint8 E8M0 bytes, got {escale.dtype}")
    K, N = qweight.shape[0] * 8, qweight.shape[1]
    if escale.shape != (K // 32, N) or K % 32:
        raise ValueError(f"escale shape {tuple(escale.shape)} does not match (K/32, N)")
    return K, N


def _mx_layer(fn_name: str, x, qweight, escale, out, workspace, stream):
    torch = _torch()
    K, N = _mx_weights(qweight, escale)
    _cuda_contig("x", x)
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise TypeError("x must be a 2-D torch.bfloat16 tensor")
    M = x.shape[0]
    if x.shape[1] != K:
        raise ValueError(f"x has {x.shape[1]} columns, qweight holds K = {K} rows")
    out = _out("out", out, (M, N), torch.bfloat16, x.device)
    lib = load_library()
    sp = _stream_ptr(stream)
    if workspace is None:
        op = OP_GEMM if fn_name == "w4a16_mxfp4_gemm" else OP_GEMV
        need = lib.w4a16_workspace_bytes(op, M, N, K, 32)
        workspace = _cached_workspace(need, x.device, stream, op) if need else None
    ws_ptr, ws_bytes = _workspace_args(workspace)
    if fn_name == "w4a16_mxfp4_gemm":
        _check(fn_name, lib.w4a16_mxfp4_gemm(x.data_ptr(), qweight.data_ptr(), escale.data_ptr(), out.data_ptr(),
                                              M, N, K, ws_ptr, ws_bytes, sp))
        return out
    _check(fn_name, lib.w4a16_mxfp4_gemv(x.data_ptr(), qweight.data_ptr(), escale.data_ptr(), out.data_ptr(),
                                          M, N, K, ws_ptr, ws_bytes, sp))
    return out


def mxfp4_gemv(x, qweight, escale, out=None, workspace=None, stream=None):
    """Decode path for MXFP4 weights (E2M1 codes in `qweight`, E8M0 bytes
    `escale` [K/32, N]); x bf16 [M, K] with 1 <= M <= 16. Returns bf16 y [M, N]."""
    return _mx_layer("w4a16_mxfp4_gemv", x, qweight, escale, out, workspace, stream)


def mxfp4_gemm(x, qweight, escale, out=None, workspace=None, stream=None):
    """Prefill path for MXFP4 weights (any M >= 1, tcgen05). Returns bf16 y [M, N]."""
    return _mx_layer("w4a16_mxfp4_gemm", x, qweight, escale, out, workspace, stream)


def mxfp4_dequant(qweight, escale, out=None, stream=None):
    """Dense bf16 copy W[k, n] = E2M1(q[k, n]) * 2^(e[k/32, n] - 127), [K, N]."""
    torch = _torch()
    K, N = _mx_weights(qweight, escale)
    out = _out("out", out, (K, N), torch.bfloat16, qweight.device)
    _check("w4a16_mxfp4_dequant", load_library().w4a16_mxfp4_dequant(qweight.data_ptr(), escale.data_ptr(),
                                                                       out.data_ptr(), N, K, _stream_ptr(stream)))
    return out


def mxfp4_scale_shape(rows: int, cols: int):
    """Shape of the exponent bytes of a row-layout operand [rows, cols]: tiles of
    128 rows x 4 blocks, [row tile, block tile, row % 32, row // 32 % 4, block % 4]."""
    return (-(-rows // 128), -(-cols // 128), 32, 4, 4)


def mxfp4_quantize(x, dim: int, out=None, stream=None):
    """Quantise x (float16, bfloat16 or float32) to MXFP4 in blocks of 32 along
    `dim`. Returns (codes, escale); `out` may give both to write into.

    dim 0: x [K, N], or [E, K, N] for a stack of matrices -> int32 [(E,) K/8, N]
           and uint8 [(E,) K/32, N], the weight layout of mxfp4_gemv, mxfp4_gemm
           and mxfp4_moe.
    dim 1: x [R, K] -> int32 [R, K/8] and uint8 mxfp4_scale_shape(R, K), the row
           layout of mxfp4_matmul."""
    torch = _torch()
    _cuda_contig("x", x)
    dt = _dtype_code(x.dtype)
    shape = x.shape
    if dim == 1 and len(shape) == 2:
        rows, cols = shape
        K = cols
        shapes = (rows, K // 8), mxfp4_scale_shape(rows, cols)
    elif dim == 0 and len(shape) in (2, 3):
        K, cols = shape[-2:]
        rows = K if len(shape) == 2 else shape[0] * K
        shapes = (*shape[:-2], K // 8, cols), (*shape[:-2], K // 32, cols)
    else:
        raise ValueError(f"x must be 2-D (or 3-D with dim 0) and dim 0 or 1, got {len(shape)}-D and dim {dim}")
    if K % 32 or not rows or not cols:
        raise ValueError(f"x must hold whole blocks of 32 along dim {dim}, got shape {tuple(shape)}")
    codes, escale = (None, None) if out is None else out
    device = x.device
    codes = _out("codes", codes, shapes[0], torch.int32, device, stream)
    escale = _out("escale", escale, shapes[1], torch.uint8, device, stream)
    st = load_library().w4a16_mxfp4_quantize(x.data_ptr(), codes.data_ptr(), escale.data_ptr(), rows, cols, dim, dt,
                                             _stream_ptr(stream))
    _check("w4a16_mxfp4_quantize", st)
    return codes, escale


def _mx_rows(name: str, codes, escale):
    """Checks a row-layout operand, returns its rows and K."""
    torch = _torch()
    _cuda_contig(name, codes)
    _cuda_contig(name + " scales", escale, codes.get_device())
    shape = codes.shape
    if len(shape) != 2 or codes.dtype != torch.int32:
        raise TypeError(f"{name} must be a 2-D torch.int32 tensor of codes")
    R, words = shape
    K = words * 8
    if escale.dtype != torch.uint8 or escale.shape != (-(-R // 128), -(-K // 128), 32, 4, 4):
        raise ValueError(f"{name} scales must be torch.uint8 {mxfp4_scale_shape(R, K)}, got {escale.dtype} "
                         f"{tuple(escale.shape)}")
    return R, K


def mxfp4_dequant_rows(codes, escale, out=None, stream=None):
    """Dense bf16 copy [R, K] of the row layout."""
    R, K = _mx_rows("codes", codes, escale)
    out = _out("out", out, (R, K), _torch().bfloat16, codes.device, stream)
    st = load_library().w4a16_mxfp4_dequant_rows(codes.data_ptr(), escale.data_ptr(), out.data_ptr(), R, K,
                                                 _stream_ptr(stream))
    _check("w4a16_mxfp4_dequant_rows", st)
    return out


def mxfp4_tile_scales(escale, out=None, stream=None):
    """Exponent bytes [R, K/32], one row after the other, to the tiles of the row layout."""
    torch = _torch()
    _cuda_contig("escale", escale)
    if escale.dim() != 2 or escale.dtype != torch.uint8:
        raise TypeError("escale must be a 2-D torch.uint8 tensor")
    R, K = escale.shape[0], escale.shape[1] * 32
    out = _out("out", out, mxfp4_scale_shape(R, K), torch.uint8, escale.device, stream)
    st = load_library().w4a16_mxfp4_tile_scales(escale.data_ptr(), out.data_ptr(), R, K, _stream_ptr(stream))
    _check("w4a16_mxfp4_tile_scales", st)
    return out


_workspace_needs = {}


def _workspace(given, op, query, shape, device, stream):
    """(address, bytes) of the caller's workspace or the binding's own, which
    needs query(*shape) bytes on the current device; the sizes of the last few
    hundred shapes are kept. A size of 0 is not: the library also answers so
    where the query itself fails."""
    if given is None:
        key = (op, device.index, shape)
        need = _workspace_needs.get(key)
        if need is None:
            need = int(query(*shape))
            if need:
                if len(_workspace_needs) >= 512:
                    _workspace_needs.clear()
                _workspace_needs[key] = need
        if not need:
            return 0, 0
        given = _cached_workspace(need, device, stream, op)
        return given.data_ptr(), given.numel()
    return _workspace_args(given)


def mxfp4_matmul(a, a_scale, b, b_scale, out_dtype=None, out=None, workspace=None, stream=None):
    """y = A @ B.T of two row-layout operands: A [M, K] (activations through
    mxfp4_quantize(x, 1)) and B [N, K] (a weight, one output feature per row).
    4-bit tensor-core product, FP32 sums; returns y [M, N] in `out_dtype`
    (bfloat16 unless given; float16 and float32 too)."""
    M, K = _mx_rows("a", a, a_scale)
    N, Kb = _mx_rows("b", b, b_scale)
    if K != Kb:
        raise ValueError(f"a has K = {K}, b has K = {Kb}")
    if out_dtype is None:
        out_dtype = _torch().bfloat16 if out is None else out.dtype
    dt = _dtype_code(out_dtype)
    lib = load_library()
    device = a.device
    out = _out("out", out, (M, N), out_dtype, device, stream)
    if M <= 32:   # tiles shared between thread blocks only there
        ws_ptr, ws_bytes = _workspace(workspace, OP_MXFP4_MATMUL, lib.w4a16_workspace_bytes,
                                      (OP_MXFP4_MATMUL, M, N, K, 32), device, stream)
    else:
        ws_ptr, ws_bytes = _workspace_args(workspace)
    st = lib.w4a16_mxfp4_matmul(a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(), out.data_ptr(),
                                M, N, K, dt, ws_ptr, ws_bytes, _stream_ptr(stream))
    _check("w4a16_mxfp4_matmul", st)
    return out


def mxfp4_moe(x, router, w13, e13, w2, e2, top_k: int, renormalize: bool = True, out=None, workspace=None,
              stream=None):
    """Mixture-of-experts layer with MXFP4 expert weights for 1..64 tokens, in one
    kernel: router product, softmax, the top_k experts of each token (their
    weights divided by their sum where `renormalize`), gate and up products,
    SwiGLU, down product and the weighted sum.

    x bf16 [T, H], router bf16 [E, H]; w13 int32 [E, H/8, 2 I] with e13 uint8
    [E, H/32, 2 I] (gate columns, then up columns) and w2 int32 [E, I/8, H] with
    e2 uint8 [E, I/32, H], as mxfp4_quantize(w, 0) makes them of [E, H, 2 I] and
    [E, I, H]. Returns y bf16 [T, H]."""
    torch = _torch()
    bf16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    _cuda_contig("x", x)
    current = x.get_device()
    for name, t, dtype, dims in (("x", x, bf16, 2), ("router", router, bf16, 2), ("w13", w13, i32, 3),
                                 ("e13", e13, u8, 3), ("w2", w2, i32, 3), ("e2", e2, u8, 3)):
        _cuda_contig(name, t, current)
        if t.dim() != dims or t.dtype != dtype:
            raise TypeError(f"{name} must be a {dims}-D {dtype} tensor, got {t.dim()}-D {t.dtype}")
    T, H = x.shape
    E, I = w2.shape[0], w2.shape[1] * 8
    for name, t, shape in (("router", router, (E, H)), ("w13", w13, (E, H // 8, 2 * I)),
                           ("e13", e13, (E, H // 32, 2 * I)), ("w2", w2, (E, I // 8, H)), ("e2", e2, (E, I // 32, H))):
        if t.shape != shape:
            raise ValueError(f"{name} shape {tuple(t.shape)} does not match {shape}")
    lib = load_library()
    device = x.device
    out = _out("out", out, (T, H), bf16, device, stream)
    ws_ptr, ws_bytes = _workspace(workspace, "mxfp4_moe", lib.w4a16_mxfp4_moe_workspace_bytes, (T, E, top_k, H, I),
                                  device, stream)
    st = lib.w4a16_mxfp4_moe(x.data_ptr(), router.data_ptr(), w13.data_ptr(), e13.data_ptr(), w2.data_ptr(),
                             e2.data_ptr(), out.data_ptr(), T, E, top_k, H, I, 1 if renormalize else 0, ws_ptr,
                             ws_bytes, _stream_ptr(stream))
    _check("w4a16_mxfp4_moe", st)
    return out


def int8_quantize(x, out=None, stream=None):
    """Quantise the rows of x [R, K] (float16, bfloat16 or float32) to int8, with
    one scale per row: scale = max |x| / 127, codes to nearest even. Returns
    (codes int8 [R, K], scale float32 [R]); `out` may give both to write into.
    Activations: a row per token. A weight: [N, K], a row per output channel."""
    torch = _torch()
    if not _here(x, _device_now()):
        _cuda_contig("x", x)
    dt = _dtype_code(x.dtype)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be 2-D, got {len(shape)}-D")
    R, K = shape
    if out is None and stream is None:
        device = x.device
        codes = torch.empty(shape, dtype=torch.int8, device=device)
        scale = torch.empty((R,), dtype=torch.float32, device=device)
    else:
        codes, scale = (None, None) if out is None else out
        codes = _out("codes", codes, shape, torch.int8, x.device, stream)
        scale = _out("scale", scale, (R,), torch.float32, x.device, stream)
    st = load_library().w4a16_int8_quantize(x.data_ptr(), codes.data_ptr(), scale.data_ptr(), R, K, dt,
                                                      _stream_ptr(stream))
    if st:
        _check("w4a16_int8_quantize", st)
    return codes, scale


def _device_now() -> int:
    """The current device; no device's number where there is none to ask."""
    try:
        return _current_device()
    except RuntimeError:
        return -2


def _here(t, current: int) -> bool:
    """Whether a tensor is dense and on the current device."""
    return t.get_device() == current and t.is_contiguous()


def _int8_rows(name: str, codes, scale, current: int):
    """Checks int8 rows and their scales, returns rows and K."""
    if not (_here(codes, current) and _here(scale, current)):
        _cuda_contig(name, codes)
        _cuda_contig(name + " scale", scale)
    shape = codes.shape
    if codes.dtype != _torch_module.int8 or len(shape) != 2:
        raise TypeError(f"{name} must be a 2-D torch.int8 tensor of codes")
    R, K = shape
    if scale.dtype != _torch_module.float32 or scale.shape != (R,):
        raise ValueError(f"{name} scale must be torch.float32 ({R},), got {scale.dtype} {tuple(scale.shape)}")
    return R, K


def int8_dequant(codes, scale, out_dtype=None, out=None, stream=None):
    """Dense copy [R, K] of int8 rows: code * scale, in `out_dtype` (bfloat16
    unless given; float16 and float32 too)."""
    torch = _torch()
    R, K = _int8_rows("codes", codes, scale, _device_now())
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    dt = _dtype_code(out_dtype)
    if out is None and stream is None:
        out = torch.empty((R, K), dtype=out_dtype, device=codes.device)
    else:
        out = _out("out", out, (R, K), out_dtype, codes.device, stream)
    st = load_library().w4a16_int8_dequant(codes.data_ptr(), scale.data_ptr(), out.data_ptr(), R, K, dt,
                                                     _stream_ptr(stream))
    if st:
        _check("w4a16_int8_dequant", st)
    return out


def int8_matmul(a, a_scale, b, b_scale, out_dtype=None, out=None, workspace=None, stream=None):
    """y = (A @ B.T) * a_scale[:, None] * b_scale of two int8 operands: A [M, K]
    (activations through int8_quantize) and B [N, K] (a weight, one output channel
    per row). Returns y [M, N] in `out_dtype` (bfloat16 unless given; float16 and
    float32 too). Sums are exact while every partial sum stays within 2^24; past
    that more than a few rows are summed in FP32, and y of a row may depend on M."""
    torch = _torch()
    current = _device_now()
    M, K = _int8_rows("a", a, a_scale, current)
    N, Kb = _int8_rows("b", b, b_scale, current)
    if K != Kb:
        raise ValueError(f"a has K = {K}, b has K = {Kb}")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    dt = _dtype_code(out_dtype)
    lib = load_library()
    device = a.device
    if out is None and stream is None:
        out = torch.empty((M, N), dtype=out_dtype, device=device)
    else:
        out = _out("out", out, (M, N), out_dtype, device, stream)
    if workspace is None and M <= 4:   # dot products: none
        ws_ptr = ws_bytes = 0
    else:
        ws_ptr, ws_bytes = _workspace(workspace, "int8_matmul", lib.w4a16_int8_matmul_workspace_bytes, (M, N, K),
                                      device, stream)
    st = lib.w4a16_int8_matmul(a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(), out.data_ptr(), M,
                               N, K, dt, ws_ptr, ws_bytes, _stream_ptr(stream))
    if st:
        _check("w4a16_int8_matmul", st)
    return out


def _norm_vector(name: str, t, dtype, H: int, current: int) -> int:
    """Address of a vector over the channels, checked; 0 for none."""
    if t is None:
        return 0
    if not _here(t, current):
        _cuda_contig(name, t)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (H,):
        raise ValueError(f"{name} shape {tuple(t.shape)} does not match {(H,)}")
    return t.data_ptr()


def block_norm(residual, weight=None, h=None, after=None, gate=None, scale: float = 1.0, eps: float = 1e-6,
               quantize: bool = False, out=None, stream=None):
    """The step between two blocks: norm after a block, gate, scaled residual
    update, norm before the next block, in one kernel.

        u  = h * rsqrt(mean(h^2) + eps) * after     (u = h without `after`)
        r' = residual + scale * gate * u            (r' = residual without `h`)
        y  = r' * rsqrt(mean(r'^2) + eps) * weight

    residual [T, H] in h's dtype or float32; h, gate, after [H], weight [H] in one
    dtype (float16, bfloat16 or float32); gate [H] (a factor per channel), [T, 1]
    (per token) or [T, H]. Returns (r', y), with y in that dtype, or with `quantize`
    (r', codes, scale), y as int8_quantize makes it. Without `weight` it returns
    r' alone; without `h`, r' is `residual` itself. `out` may give the outputs to
    write into, as a tuple in the order of the result (r' may be `residual`)."""
    torch = _torch()
    current = _device_now()
    if not _here(residual, current):
        _cuda_contig("residual", residual)
    shape = residual.shape
    if len(shape) != 2:
        raise ValueError(f"residual must be 2-D, got {len(shape)}-D")
    T, H = shape
    if h is not None:
        dtype = h.dtype
        if not _here(h, current):
            _cuda_contig("h", h)
        if h.shape != shape:
            raise ValueError(f"h shape {tuple(h.shape)} does not match {tuple(shape)}")
        h_ptr = h.data_ptr()
    else:
        if weight is None:
            raise ValueError("h or weight must be given")
        if after is not None or gate is not None:
            raise ValueError("after and gate need h")
        dtype, h_ptr = weight.dtype, 0
    if quantize and weight is None:
        raise ValueError("quantize needs weight")
    dt, rdt = _dtype_code(dtype), _dtype_code(residual.dtype)
    if rdt != dt and rdt != F32:
        raise TypeError(f"residual must be {dtype} or float32, got {residual.dtype}")
    weight_ptr = _norm_vector("weight", weight, dtype, H, current)
    after_ptr = _norm_vector("after", after, dtype, H, current)
    gate_ptr, kind = 0, GATE_CHANNEL
    if gate is not None:
        if gate.shape == (H,):
            gate_ptr = _norm_vector("gate", gate, dtype, H, current)
        else:
            kind = GATE_ELEMENT if gate.shape == shape else GATE_TOKEN
            if kind == GATE_TOKEN and gate.shape != (T, 1):
                raise ValueError(f"gate shape {tuple(gate.shape)} is none of {(H,)}, {(T, 1)}, {(T, H)}")
            if not _here(gate, current):
                _cuda_contig("gate", gate)
            if gate.dtype != dtype:
                raise TypeError(f"gate must be {dtype}, got {gate.dtype}")
            gate_ptr = gate.data_ptr()
    y = codes = code_scale = None
    if out is None and stream is None:
        device = residual.device
        new = residual if h is None else torch.empty(shape, dtype=residual.dtype, device=device)
        if quantize:
            codes = torch.empty(shape, dtype=torch.int8, device=device)
            code_scale = torch.empty((T,), dtype=torch.float32, device=device)
        elif weight is not None:
            y = torch.empty(shape, dtype=dtype, device=device)
    else:
        outs = [None] * 3 if out is None else list(out) if isinstance(out, (tuple, list)) else [out]
        if out is not None and len(outs) != (1 if weight is None else 3 if quantize else 2):
            raise ValueError(f"out holds {len(outs)} tensors")
        device = residual.device
        if h is not None:
            new = _out("residual out", outs[0], shape, residual.dtype, device, stream)
        elif outs[0] is None or outs[0] is residual:
            new = residual
        else:
            raise ValueError("without h the residual is returned as it is")
        if quantize:
            codes = _out("codes", outs[1], shape, torch.int8, device, stream)
            code_scale = _out("scale", outs[2], (T,), torch.float32, device, stream)
        elif weight is not None:
            y = _out("y", outs[1], shape, dtype, device, stream)
    st = load_library().w4a16_block_norm(
        residual.data_ptr(), rdt, h_ptr, after_ptr, gate_ptr, kind, scale, 0 if h is None else new.data_ptr(),
        weight_ptr, eps, 0 if y is None else y.data_ptr(), 0 if codes is None else codes.data_ptr(),
        0 if codes is None else code_scale.data_ptr(), T, H, dt, _stream_ptr(stream))
    if st:
        _check("w4a16_block_norm", st)
    if weight is None:
        return new
    return (new, codes, code_scale) if quantize else (new, y)


def device_status(stream=None) -> int:
    """Synchronise the stream, return and clear the device-side error status."""
    return int(load_library().w4a16_device_status(_stream_ptr(stream)))


def selftest_wait_timeout(stream=None) -> None:
    """Launch the bounded-wait self-test (one warp waits on a barrier nothing
    completes; it gives up after about two seconds and records
    W4A16_ERR_TIMEOUT, which `device_status` then returns)."""
    _check("w4a16_selftest_wait_timeout", load_library().w4a16_selftest_wait_timeout(_stream_ptr(stream)))
