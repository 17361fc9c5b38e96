"""ctypes binding of libluce_moe (include/luce_moe.h), same names as the C ABI.

Argument marshalling only: each function checks that its tensors are CUDA,
contiguous and of the right dtype, passes ``data_ptr()`` values and the
current torch stream (or the one given), and raises :class:`LuceError` when
the library returns a status other than ``LUCE_OK``.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback: if the
library has not been built, the first call raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from .build import LIB as LIB_PATH
from .build import call_path

LUCE_OK = 0
LUCE_ERR_INVALID_ARG = 1
LUCE_ERR_UNSUPPORTED = 2
LUCE_ERR_CUDA = 3
LUCE_F32 = 0
LUCE_BF16 = 1
LUCE_F16 = 2
LUCE_FAULT_BAD_ID = 0x1
LUCE_FAULT_TIMEOUT = 0x2
LUCE_FAULT_DESYNC = 0x4

_LIB = None
_fast = None  # the call module, loaded with the library; None where there is none


class LuceError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it was not built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run quantized_moe_decode_luce_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        sigs = {
            "luce_route_topk": [P, P, i32, i32, i32, P, P, P],
            "luce_quantize_q8_1": [P, i32, i32, P, P],
            "luce_moe_group": [P, i32, i32, i32, P, P, P, P],
            "luce_moe_glu_pair": [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P, i32, P],
            "luce_moe_prep": [P, P, P, i32, i32, i32, i32, P, P, P, P, P, P, P],
            "luce_moe_layer": [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P, P, P, P, P, P, P, P,
                               P, sz, P],
            "luce_moe_down_combine": [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, P, i32, P],
            "luce_argmax": [P, i32, i64, P, P, P, sz, P],
            "luce_argmax_noalloc": [P, i32, i64, P, P, P],
            "luce_argmax_shard": [P, i32, i64, i64, P, P, P, sz, P],
            "luce_argmax_pick": [P, P, i32, i32, P, P, P],
            "luce_rmsnorm_router": [P, P, f32, P, i32, i32, i32, P, P, P],
            "luce_add_rmsnorm_router": [P, P, P, P, f32, P, i32, i32, i32, P, P, P],
            "luce_ep_mask": [P, i64, i32, i32, P, P],
            "luce_add_f32": [P, P, P, i64, P],
            "luce_moe_glu_q4k": [P, P, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P, P],
            "luce_moe_down_combine_q4k": [P, P, P, P, P, i32, i32, i32, i32, i32, P, P],
            "luce_quantize_i8": [P, i32, i32, i32, P, P, P],
            "luce_rmsnorm_i8": [P, i32, P, f32, i32, i32, P, P, P],
            "luce_add_rmsnorm_i8": [P, P, P, i32, P, f32, i32, i32, P, P, P],
            "luce_linear_i8": [P, P, P, P, P, i32, i32, i32, P, i32, i64, P],
            "luce_linear_i8_plan": [i32, i32, i32, i32, P],
            "luce_logits_process": [P, i32, i32, i64, i64, P, i64, P, P, P, P, P, P, P, i32, P, i32, i64, P, P, i64,
                                    P],
        }
        for name, args in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.luce_set_pdl.argtypes = [i32]
        L.luce_set_pdl.restype = ctypes.c_int
        L.luce_moe_layer_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.luce_moe_layer_workspace_bytes.restype = sz
        L.luce_argmax_workspace_bytes.argtypes = [i32, i64]
        L.luce_argmax_workspace_bytes.restype = sz
        L.luce_status_string.argtypes = [ctypes.c_int]
        L.luce_status_string.restype = ctypes.c_char_p
        L.luce_get_fault.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.luce_get_fault.restype = ctypes.c_int
        L.luce_version.argtypes = []
        L.luce_version.restype = ctypes.c_int
        _load_call_module(L)
        _LIB = L
    return _LIB


def _load_call_module(L) -> None:
    """The module that makes the common calls of the int8 head without Python in between.  The code
    below serves every call without it, a few microseconds of host time slower."""
    global _fast
    try:
        loader = importlib.machinery.ExtensionFileLoader("luce_call", call_path())
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("luce_call", loader))
        loader.exec_module(module)
    except (ImportError, OSError) as e:
        warnings.warn(f"no call module (run quantized_moe_decode_luce_gb300.build.build()): {e}", RuntimeWarning,
                      stacklevel=3)
        return
    module.bind(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
        "luce_quantize_i8", "luce_rmsnorm_i8", "luce_add_rmsnorm_i8", "luce_linear_i8", "luce_logits_process")))
    _fast = module


def status_string(status: int) -> str:
    return lib().luce_status_string(int(status)).decode()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t, dtype=None, name="tensor") -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _check(fn: str, status: int) -> None:
    if status != LUCE_OK:
        raise LuceError(fn, status)


u8, i32, f32 = torch.uint8, torch.int32, torch.float32


def luce_route_topk(logits, bias, k: int, ids, weights, stream=None) -> None:
    T, E = logits.shape
    _check("luce_route_topk", lib().luce_route_topk(
        _ptr(logits, f32, "logits"), _ptr(bias, f32, "bias"), T, E, k, _ptr(ids, i32, "ids"),
        _ptr(weights, f32, "weights"), _stream(stream)))


def luce_quantize_q8_1(x, xq, stream=None) -> None:
    T, K = x.shape
    _check("luce_quantize_q8_1", lib().luce_quantize_q8_1(
        _ptr(x, f32, "x"), T, K, _ptr(xq, u8, "xq"), _stream(stream)))


def luce_moe_group(ids, E: int, counts, offsets, routes, stream=None) -> None:
    T, k = ids.shape
    _check("luce_moe_group", lib().luce_moe_group(
        _ptr(ids, i32, "ids"), T, k, E, _ptr(counts, i32, "counts"), _ptr(offsets, i32, "offsets"),
        _ptr(routes, i32, "routes"), _stream(stream)))


def luce_moe_glu_pair(w_gate, w_up, ws_gate, ws_up, xq, offsets, routes, T: int, k: int, E: int, H: int, I: int,
                      clamp: float, h, hq, variant: int = 0, stream=None) -> None:
    _check("luce_moe_glu_pair", lib().luce_moe_glu_pair(
        _ptr(w_gate, u8, "w_gate"), _ptr(w_up, u8, "w_up"), _ptr(ws_gate, u8, "ws_gate"), _ptr(ws_up, u8, "ws_up"),
        _ptr(xq, u8, "xq"), _ptr(offsets, i32, "offsets"), _ptr(routes, i32, "routes"), T, k, E, H, I,
        float(clamp), _ptr(h, f32, "h"), _ptr(hq, u8, "hq"), variant, _stream(stream)))


def luce_moe_prep(logits, bias, x, k: int, ids, weights, xq, counts, offsets, routes, stream=None) -> None:
    T, E = logits.shape
    H = x.shape[1]
    _check("luce_moe_prep", lib().luce_moe_prep(
        _ptr(logits, f32, "logits"), _ptr(bias, f32, "bias"), _ptr(x, f32, "x"), T, E, k, H, _ptr(ids, i32, "ids"),
        _ptr(weights, f32, "weights"), _ptr(xq, u8, "xq"), _ptr(counts, i32, "counts"),
        _ptr(offsets, i32, "offsets"), _ptr(routes, i32, "routes"), _stream(stream)))


def luce_moe_layer_workspace_bytes(T: int, k: int, H: int, I: int) -> int:
    return int(lib().luce_moe_layer_workspace_bytes(T, k, H, I))


def luce_moe_layer(logits, bias, x, k: int, I: int, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, clamp: float,
                   ids, weights, xq, counts, offsets, routes, h, hq, out, workspace, stream=None) -> None:
    """The whole layer in one launch; `workspace` is a uint8 CUDA tensor of at
    least luce_moe_layer_workspace_bytes(T, k, H, I) bytes, all zero before
    the first call (the library keeps it consistent)."""
    T, E = logits.shape
    H = x.shape[1]
    if workspace is None:
        raise ValueError("workspace is required")
    _check("luce_moe_layer", lib().luce_moe_layer(
        _ptr(logits, f32, "logits"), _ptr(bias, f32, "bias"), _ptr(x, f32, "x"), _ptr(w_gate, u8, "w_gate"),
        _ptr(w_up, u8, "w_up"), _ptr(w_down, u8, "w_down"), _ptr(ws_gate, u8, "ws_gate"), _ptr(ws_up, u8, "ws_up"),
        _ptr(ws_down, u8, "ws_down"), T, E, k, H, I, float(clamp), _ptr(ids, i32, "ids"),
        _ptr(weights, f32, "weights"), _ptr(xq, u8, "xq"), _ptr(counts, i32, "counts"),
        _ptr(offsets, i32, "offsets"), _ptr(routes, i32, "routes"), _ptr(h, f32, "h"), _ptr(hq, u8, "hq"),
        _ptr(out, f32, "out"), _ptr(workspace, u8, "workspace"), workspace.numel(), _stream(stream)))


def luce_set_pdl(enable: bool) -> None:
    _check("luce_set_pdl", lib().luce_set_pdl(1 if enable else 0))


def luce_moe_down_combine(w_down, ws_down, hq, ids, weights, offsets, routes, T: int, k: int, E: int, H: int,
                          I: int, out, variant: int = 0, stream=None) -> None:
    _check("luce_moe_down_combine", lib().luce_moe_down_combine(
        _ptr(w_down, u8, "w_down"), _ptr(ws_down, u8, "ws_down"), _ptr(hq, u8, "hq"), _ptr(ids, i32, "ids"),
        _ptr(weights, f32, "weights"), _ptr(offsets, i32, "offsets"), _ptr(routes, i32, "routes"),
        T, k, E, H, I, _ptr(out, f32, "out"), variant, _stream(stream)))


def luce_argmax_workspace_bytes(R: int, V: int) -> int:
    return int(lib().luce_argmax_workspace_bytes(R, V))


def luce_argmax(logits, idx, val, workspace, stream=None) -> None:
    R, V = logits.shape
    _check("luce_argmax", lib().luce_argmax(
        _ptr(logits, f32, "logits"), R, V, _ptr(idx, i32, "idx"), _ptr(val, f32, "val"),
        _ptr(workspace, u8, "workspace"), workspace.numel() if workspace is not None else 0, _stream(stream)))


def luce_argmax_noalloc(logits, idx, val, stream=None) -> None:
    """The argmax with the library's own fixed scratch (no allocation)."""
    R, V = logits.shape
    _check("luce_argmax_noalloc", lib().luce_argmax_noalloc(
        _ptr(logits, f32, "logits"), R, V, _ptr(idx, i32, "idx"), _ptr(val, f32, "val"), _stream(stream)))


def luce_argmax_shard(logits, v0: int, idx, val, workspace, stream=None) -> None:
    """Argmax of a vocabulary shard whose column 0 is column v0 of the whole vocabulary."""
    R, Vs = logits.shape
    _check("luce_argmax_shard", lib().luce_argmax_shard(
        _ptr(logits, f32, "logits"), R, Vs, int(v0), _ptr(idx, i32, "idx"), _ptr(val, f32, "val"),
        _ptr(workspace, u8, "workspace"), workspace.numel() if workspace is not None else 0, _stream(stream)))


def luce_argmax_pick(vals, idxs, idx, val, stream=None) -> None:
    """vals [S, R] fp32, idxs [S, R] int32 (the shards' results) -> idx [R], val [R]."""
    S, R = vals.shape
    _check("luce_argmax_pick", lib().luce_argmax_pick(
        _ptr(vals, f32, "vals"), _ptr(idxs, i32, "idxs"), S, R, _ptr(idx, i32, "idx"), _ptr(val, f32, "val"),
        _stream(stream)))


def luce_rmsnorm_router(x, gamma, eps: float, w_router, xn, logits, stream=None) -> None:
    """x [T, H], gamma [H], w_router [E, H] (fp32) -> xn [T, H] (or None), logits [T, E]."""
    T, H = x.shape
    E = w_router.shape[0]
    _check("luce_rmsnorm_router", lib().luce_rmsnorm_router(
        _ptr(x, f32, "x"), _ptr(gamma, f32, "gamma"), float(eps), _ptr(w_router, f32, "w_router"), T, E, H,
        _ptr(xn, f32, "xn"), _ptr(logits, f32, "logits"), _stream(stream)))


def luce_add_rmsnorm_router(x, residual, x_sum, gamma, eps: float, w_router, xn, logits, stream=None) -> None:
    """x, residual [T, H] -> x_sum = x + residual (or None), then luce_rmsnorm_router of the sum."""
    T, H = x.shape
    if tuple(residual.shape) != (T, H):
        raise ValueError("residual must have x's shape")
    E = w_router.shape[0]
    _check("luce_add_rmsnorm_router", lib().luce_add_rmsnorm_router(
        _ptr(x, f32, "x"), _ptr(residual, f32, "residual"), _ptr(x_sum, f32, "x_sum"), _ptr(gamma, f32, "gamma"),
        float(eps), _ptr(w_router, f32, "w_router"), T, E, H, _ptr(xn, f32, "xn"), _ptr(logits, f32, "logits"),
        _stream(stream)))


def luce_ep_mask(ids, e0: int, e1: int, ids_out, stream=None) -> None:
    _check("luce_ep_mask", lib().luce_ep_mask(
        _ptr(ids, i32, "ids"), ids.numel(), int(e0), int(e1), _ptr(ids_out, i32, "ids_out"), _stream(stream)))


def luce_add_f32(a, b, out, stream=None) -> None:
    if a.numel() != b.numel() or a.numel() != out.numel():
        raise ValueError("a, b and out must have the same number of elements")
    _check("luce_add_f32", lib().luce_add_f32(
        _ptr(a, f32, "a"), _ptr(b, f32, "b"), _ptr(out, f32, "out"), a.numel(), _stream(stream)))


def luce_moe_glu_q4k(w_gate, w_up, ws_gate, ws_up, xq, ids, E: int, H: int, I: int, clamp: float, h, hq=None,
                     stream=None) -> None:
    """Q4_K gate/up pair + SwiGLU -> h, and its q8_1 blocks -> hq when given."""
    T, k = ids.shape
    _check("luce_moe_glu_q4k", lib().luce_moe_glu_q4k(
        _ptr(w_gate, u8, "w_gate"), _ptr(w_up, u8, "w_up"), _ptr(ws_gate, u8, "ws_gate"), _ptr(ws_up, u8, "ws_up"),
        _ptr(xq, u8, "xq"), _ptr(ids, i32, "ids"), T, k, E, H, I, float(clamp), _ptr(h, f32, "h"),
        _ptr(hq, u8, "hq"), _stream(stream)))


def luce_moe_down_combine_q4k(w_down, ws_down, hq, ids, weights, E: int, H: int, I: int, out, stream=None) -> None:
    """Q4_K down product + masked route-weighted combine -> out."""
    T, k = ids.shape
    _check("luce_moe_down_combine_q4k", lib().luce_moe_down_combine_q4k(
        _ptr(w_down, u8, "w_down"), _ptr(ws_down, u8, "ws_down"), _ptr(hq, u8, "hq"), _ptr(ids, i32, "ids"),
        _ptr(weights, f32, "weights"), T, k, E, H, I, _ptr(out, f32, "out"), _stream(stream)))


# ----------------------------------------------------------------------------- int8 decode head
# These entry points check shapes as well, and run on the device that holds
# their tensors, on its current stream unless one is given.  The common call
# (that stream, the current device, nothing to object to) goes through the call
# module in one step; it leaves every other call (-1) to the code here.
_DTYPE = {torch.float32: LUCE_F32, torch.bfloat16: LUCE_BF16, torch.float16: LUCE_F16}
_FLOATS = frozenset(_DTYPE)
_F32, _I8, _I32, _WORDS = frozenset({torch.float32}), frozenset({torch.int8}), frozenset({torch.int32}), \
    frozenset({torch.int32, torch.uint32})


# torch's own call behind torch.cuda.current_stream(dev).cuda_stream, without
# the Stream object around it (0.1 against 2.9 us, of a call of 9)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(t, dtypes, shape, dev, name, rows=False):
    """Raises what is wrong with `t`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    raise ValueError(f"{name} must have contiguous rows" if rows else f"{name} must be contiguous")


def _addr(t, dtypes, shape, dev, name) -> int:
    """data_ptr of a contiguous CUDA tensor of one of `dtypes`, of `shape`, on device `dev`."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, dtypes, shape, dev, name)


def _rows(t, dtypes, shape, dev, name) -> tuple[int, int]:
    """(data_ptr, row stride) of a CUDA matrix whose rows are contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return t.data_ptr(), shape[1]
        step, inner = t.stride()
        if inner == 1 or shape[1] == 1:
            return t.data_ptr(), (step if shape[0] > 1 else shape[1])
    _refuse(t, dtypes, shape, dev, name, rows=True)


def _matrix(t, name) -> tuple[int, int, int]:
    """(rows, columns, device) of a CUDA matrix."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    R, C = t.shape
    return R, C, t.get_device()


def _call(fn: str, dev: int, stream, *args) -> None:
    """The library call on device `dev`, on `stream` or the device's current stream."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call(fn, dev, stream, *args)
    if stream is None:
        s = _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != dev:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{dev}")
        s = stream.cuda_stream
    else:
        s = int(stream)
    status = getattr(_LIB or lib(), fn)(*args, s)
    if status != LUCE_OK:
        raise LuceError(fn, status)


def luce_quantize_i8(x, q, scale, stream=None) -> None:
    """x [T, H] fp32, bf16 or fp16 -> q [T, H] int8, scale [T] fp32 (q * scale stands for x)."""
    if stream is None and _fast is not None:
        status = _fast.quantize_i8(x, q, scale)
        if status >= 0:
            return _check("luce_quantize_i8", status)
    T, H, dev = _matrix(x, "x")
    _call("luce_quantize_i8", dev, stream, _addr(x, _FLOATS, (T, H), dev, "x"), _DTYPE[x.dtype], T, H,
          _addr(q, _I8, (T, H), dev, "q"), _addr(scale, _F32, (T,), dev, "scale"))


def luce_rmsnorm_i8(x, gamma, eps: float, q, scale, stream=None) -> None:
    """x [T, H], gamma [H] fp32 -> the int8 codes and scales of the RMS norm of x."""
    if stream is None and _fast is not None:
        status = _fast.rmsnorm_i8(x, gamma, eps, q, scale)
        if status >= 0:
            return _check("luce_rmsnorm_i8", status)
    T, H, dev = _matrix(x, "x")
    _call("luce_rmsnorm_i8", dev, stream, _addr(x, _FLOATS, (T, H), dev, "x"), _DTYPE[x.dtype],
          _addr(gamma, _F32, (H,), dev, "gamma"), eps, T, H, _addr(q, _I8, (T, H), dev, "q"),
          _addr(scale, _F32, (T,), dev, "scale"))


def luce_add_rmsnorm_i8(x, residual, x_sum, gamma, eps: float, q, scale, stream=None) -> None:
    """x, residual [T, H] of one type -> x_sum = x + residual (or None; may be x or residual itself),
    then luce_rmsnorm_i8 of the sum."""
    if stream is None and _fast is not None:
        status = _fast.add_rmsnorm_i8(x, residual, x_sum, gamma, eps, q, scale)
        if status >= 0:
            return _check("luce_add_rmsnorm_i8", status)
    T, H, dev = _matrix(x, "x")
    own = (x.dtype,)
    _call("luce_add_rmsnorm_i8", dev, stream, _addr(x, _FLOATS, (T, H), dev, "x"),
          _addr(residual, own, (T, H), dev, "residual"),
          None if x_sum is None else _addr(x_sum, own, (T, H), dev, "x_sum"), _DTYPE[x.dtype],
          _addr(gamma, _F32, (H,), dev, "gamma"), eps, T, H, _addr(q, _I8, (T, H), dev, "q"),
          _addr(scale, _F32, (T,), dev, "scale"))


def luce_linear_i8(xq, x_scale, wq, w_scale, bias, out, stream=None) -> None:
    """xq [T, K], wq [N, K] int8, x_scale [T], w_scale [N], bias [N] (or None) fp32 -> out [T, N]
    fp32, bf16 or fp16 (its rows may be apart: a slice of wider rows)."""
    if stream is None and _fast is not None:
        status = _fast.linear_i8(xq, x_scale, wq, w_scale, bias, out)
        if status >= 0:
            return _check("luce_linear_i8", status)
    T, K, dev = _matrix(xq, "xq")
    N = _matrix(wq, "wq")[0]
    o, ldo = _rows(out, _FLOATS, (T, N), dev, "out")
    _call("luce_linear_i8", dev, stream, _addr(xq, _I8, (T, K), dev, "xq"),
          _addr(x_scale, _F32, (T,), dev, "x_scale"), _addr(wq, _I8, (N, K), dev, "wq"),
          _addr(w_scale, _F32, (N,), dev, "w_scale"),
          None if bias is None else _addr(bias, _F32, (N,), dev, "bias"), T, N, K, o, _DTYPE[out.dtype], ldo)


def luce_linear_i8_plan(T: int, N: int, K: int, dtype=torch.float32) -> list[tuple[int, int, int, int]]:
    """What luce_linear_i8 launches for a product on the current device: (kernel, tokens of a tile,
    groups along K, channels) of one or two launches; kernel 0 is the stream of the weights, 1, 2 and 4
    are tiles of up to 64, 128 and 256 tokens."""
    plan = (ctypes.c_int * 8)()
    _check("luce_linear_i8_plan", lib().luce_linear_i8_plan(T, N, K, _DTYPE[dtype], plan))
    return [tuple(plan[i:i + 4]) for i in (0, 4) if plan[i + 3]]


def luce_logits_process(logits, out, hist=None, hist_len=None, prompt_len=None, repetition=None, frequency=None,
                        presence=None, bias_ids=None, bias_vals=None, mask=None, mask_rows=None,
                        stream=None) -> None:
    """logits [R, V] fp32, bf16 or fp16 -> out [R, V] fp32 (may be logits itself): penalties for the
    tokens of hist [R, L] (hist_len [R]; prompt_len [R] of them the prompt's), biases
    bias_ids / bias_vals [R, n], masks [M, words] of 32 tokens a word (mask_rows [R], or row r
    takes mask r).  Each group may be left out."""
    if stream is None and _fast is not None:
        status = _fast.logits_process(logits, out, hist, hist_len, prompt_len, repetition, frequency, presence,
                                      bias_ids, bias_vals, mask, mask_rows)
        if status >= 0:
            return _check("luce_logits_process", status)
    R, V, dev = _matrix(logits, "logits")
    lp, ldl = _rows(logits, _FLOATS, (R, V), dev, "logits")
    op, ldo = _rows(out, _F32, (R, V), dev, "out")
    hp, ldh, hl = None, 0, None
    if hist is not None:
        if hist_len is None:
            raise ValueError("hist needs hist_len")
        ldh = _matrix(hist, "hist")[1]
        hp, hl = _addr(hist, _I32, (R, ldh), dev, "hist"), _addr(hist_len, _I32, (R,), dev, "hist_len")
        if ldh == 0:
            hp = hl = prompt_len = None
    elif hist_len is not None or prompt_len is not None:
        raise ValueError("hist_len and prompt_len need hist")
    nb, bi, bv = 0, None, None
    if bias_ids is not None:
        nb = _matrix(bias_ids, "bias_ids")[1]
        bi, bv = _addr(bias_ids, _I32, (R, nb), dev, "bias_ids"), _addr(bias_vals, _F32, (R, nb), dev, "bias_vals")
    elif bias_vals is not None:
        raise ValueError("bias_vals needs bias_ids")
    mp, nm, ldm = None, 0, 0
    if mask is not None:
        nm, ldm = _matrix(mask, "mask")[:2]
        mp = _addr(mask, _WORDS, (nm, ldm), dev, "mask")
        # an empty tensor has no address, by which the library would know that there is a mask
        if (nm > 0 and ldm == 0) or (nm == 0 and R > 0 and mask_rows is None):
            raise LuceError("luce_logits_process", LUCE_ERR_INVALID_ARG)
    elif mask_rows is not None:
        raise ValueError("mask_rows needs mask")

    def per_row(t, dtypes, name):
        return None if t is None else _addr(t, dtypes, (R,), dev, name)

    _call("luce_logits_process", dev, stream, lp, _DTYPE[logits.dtype], R, V, ldl, hp, ldh, hl,
          per_row(prompt_len, _I32, "prompt_len"), per_row(repetition, _F32, "repetition"),
          per_row(frequency, _F32, "frequency"), per_row(presence, _F32, "presence"), bi, bv, nb, mp, nm, ldm,
          per_row(mask_rows, _I32, "mask_rows"), op, ldo)


def luce_get_fault() -> int:
    bits = ctypes.c_uint(0)
    _check("luce_get_fault", lib().luce_get_fault(ctypes.byref(bits)))
    return int(bits.value)


def luce_version() -> int:
    return int(lib().luce_version())


__all__ = ["LuceError", "lib", "status_string", "luce_route_topk", "luce_quantize_q8_1", "luce_moe_group",
           "luce_moe_glu_pair", "luce_moe_prep", "luce_moe_layer", "luce_moe_layer_workspace_bytes", "luce_set_pdl",
           "luce_moe_down_combine", "luce_argmax", "luce_argmax_workspace_bytes", "luce_argmax_noalloc",
           "luce_argmax_shard", "luce_argmax_pick", "luce_rmsnorm_router", "luce_add_rmsnorm_router", "luce_ep_mask", "luce_add_f32",
           "luce_moe_glu_q4k", "luce_moe_down_combine_q4k",
           "luce_quantize_i8", "luce_rmsnorm_i8", "luce_add_rmsnorm_i8", "luce_linear_i8", "luce_linear_i8_plan",
           "luce_logits_process", "LUCE_F32", "LUCE_BF16", "LUCE_F16",
           "luce_get_fault", "luce_version", "LUCE_OK", "LUCE_ERR_INVALID_ARG", "LUCE_ERR_UNSUPPORTED",
           "LUCE_ERR_CUDA", "LUCE_FAULT_BAD_ID", "LUCE_FAULT_TIMEOUT", "LUCE_FAULT_DESYNC"]
