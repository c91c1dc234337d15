"""Python binding of libfp8q.so: scaled FP8 quantisation and FP8 GEMM on GB300.

Argument marshalling only.  Every function here validates tensor placement,
takes raw device pointers from torch tensors, passes the current CUDA stream
and calls one C entry point declared in ``include/fp8q.h``; all arithmetic
runs in the library's CUDA kernels.  There is no CPU or PyTorch fallback: if
the library is missing or the device is not a GB300 the call raises.

The names follow the C ABI: ``fp8_amax``, ``fp8_quantize_tensor``,
``fp8_quantize_delayed``, ``fp8_quantize_tile1x128``,
``fp8_quantize_block128x128``, ``fp8_gemm`` and the role wrappers
``fp8_gemm_fprop`` / ``fp8_gemm_dgrad`` / ``fp8_gemm_wgrad``, and
``fp8_linear_autocast``; the 4-bit ``fp4_quantize``, ``fp4_dequantize``,
``fp4_gemm``, ``fp4_linear`` and ``fp4_linear_train``; ``fp8_act_forward`` /
``fp8_act_backward``, activation functions with 8-bit checkpoints; ``fp8_rmsnorm`` /
``fp8_rmsnorm_backward``; and ``fp8_quantize_experts`` with ``fp8_experts_fprop`` /
``fp8_experts_dgrad`` / ``fp8_experts_wgrad``, a linear layer per expert in MXFP8.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading
from typing import NamedTuple

import torch

E4M3 = 0
E5M2 = 1
DT_F32 = 0
DT_BF16 = 1
SCALE_TENSOR = 0
SCALE_TILE_1x128 = 1
SCALE_BLOCK_128x128 = 2
SCALE_ROW = 3
SCALE_MX_1x32 = 4
RECIPE_TENSOR_CURRENT = 0
RECIPE_TENSOR_DELAYED = 1
RECIPE_BLOCK = 2
RECIPE_MXFP8 = 3
MX_BLOCK = 32
MXFP4 = 0
NVFP4 = 1
ACT_SILU = 0
ACT_GELU = 1
ACT_GELU_TANH = 2
HISTORY_LEN = 16
HISTORY_BYTES = 80

OK = 0
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "MISALIGNED", 3: "ARCH", 4: "WORKSPACE",
                5: "TIMEOUT", 6: "CUDA", 7: "NOT_IMPLEMENTED"}

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libfp8q.so")

#: every symbol include/fp8q.h declares
EXPORTS = (
    "fp8q_status_string", "fp8q_device_status", "fp8q_device_supported",
    "fp8q_selftest_barrier_timeout", "fp8_amax",
    "fp8_quantize_tensor", "fp8_quantize_tensor_current", "fp8_quantize_delayed",
    "fp8q_history_init",
    "fp8_quantize_tile1x128", "fp8_quantize_rowwise", "fp8_quantize_mxfp8",
    "fp8q_mx_scale_bytes", "fp8_quantize_block128x128", "fp8_gemm",
    "fp8_gemm_amax", "fp8_gemm_fprop",
    "fp8_gemm_dgrad", "fp8_gemm_wgrad", "fp8_gemm_grouped", "fp8q_linear_workspace_size",
    "fp8_linear_autocast",
    "fp8_linear_autocast_noalloc", "fp8q_linear_train_workspace_size", "fp8_linear_train",
    "fp8q_linear_train_host_workspace_size", "fp8_linear_train_host",
    "fp4q_scale_bytes", "fp4_quantize", "fp4_amax", "fp4_dequantize", "fp4_gemm",
    "fp4q_linear_workspace_size", "fp4_linear",
    "fp4q_linear_train_workspace_size", "fp4_linear_train",
    "fp8_act_forward", "fp8_act_backward",
    "fp8_rmsnorm", "fp8q_rmsnorm_backward_workspace_size", "fp8_rmsnorm_backward",
    "fp8q_experts_blocks", "fp8q_experts_scale_bytes", "fp8_quantize_experts",
    "fp8_experts_fprop", "fp8_experts_dgrad", "fp8_experts_wgrad",
)


class Fp8qError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status})")


class Operand(ctypes.Structure):
    """fp8q_operand: device byte matrix [rows, K] plus its scale description."""
    _fields_ = [("data", ctypes.c_void_p), ("format", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("scale", ctypes.c_void_p),
                ("scale_stride_row", ctypes.c_int64), ("scale_stride_k", ctypes.c_int64)]


def signatures() -> dict:
    """ctypes (restype, argtypes) of every entry point, as include/fp8q.h
    declares them (tests compare the two)."""
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    OP = ctypes.POINTER(Operand)
    return {
        "fp8q_status_string": (ctypes.c_char_p, [I32]),
        "fp8q_device_status": (I32, []),
        "fp8q_device_supported": (I32, []),
        "fp8q_selftest_barrier_timeout": (I32, [P]),
        "fp8_amax": (I32, [P, I32, I64, P, P]),
        "fp8_quantize_tensor": (I32, [P, I32, I64, I64, I32, P, P, P, P, I32, P]),
        "fp8_quantize_delayed": (I32, [P, I32, I64, I64, I32, P, P, P, P, I32, P]),
        "fp8_quantize_tensor_current": (I32, [P, I32, I64, I64, I32, P, P, P, P, I32, P]),
        "fp8q_history_init": (I32, [P, P, P]),
        "fp8_quantize_tile1x128": (I32, [P, I32, I64, I64, I32, P, P, P, P, I32, P]),
        "fp8_quantize_rowwise": (I32, [P, I32, I64, I64, I32, P, P, P, P, I32, P]),
        "fp8_quantize_block128x128": (I32, [P, I32, I64, I64, I32, P, P, P, I32, P]),
        "fp8_quantize_mxfp8": (I32, [P, I32, I64, I64, I32, P, P, P, P, P]),
        "fp8q_mx_scale_bytes": (SZ, [I64, I64]),
        "fp8_gemm": (I32, [OP, OP, P, I32, I64, I64, I64, P]),
        "fp8_gemm_amax": (I32, [OP, OP, P, I32, I64, I64, I64, P, P]),
        "fp8_gemm_fprop": (I32, [OP, OP, P, I32, I64, I64, I64, P]),
        "fp8_gemm_dgrad": (I32, [OP, OP, P, I32, I64, I64, I64, P]),
        "fp8_gemm_wgrad": (I32, [OP, OP, P, I32, I64, I64, I64, P]),
        "fp8_gemm_grouped": (I32, [P, I32, I32, P]),
        "fp8q_linear_workspace_size": (SZ, [I32, I64, I64, I64]),
        "fp8_linear_autocast": (I32, [P, P, I32, I64, I64, I64, I32, P, P, P, I32, P, SZ,
                                      P]),
        "fp8_linear_autocast_noalloc": (I32, [P, P, I32, I64, I64, I64, I32, P, P, P, I32,
                                              P]),
        "fp8q_linear_train_workspace_size": (SZ, [I32, I64, I64, I64]),
        "fp8_linear_train": (I32, [P, P, P, I32, I64, I64, I64, I32, P, P, P, P, P, P, I32,
                                   P, SZ, P]),
        "fp8q_linear_train_host_workspace_size": (SZ, [I32, I32, I32, I64, I64, I64]),
        "fp8_linear_train_host": (I32, [P, P, P, I32, I64, I64, I64, I32, P, P, P, P, P, P,
                                        I32, P, SZ, P]),
        "fp4q_scale_bytes": (SZ, [I32, I64, I64]),
        "fp4_quantize": (I32, [P, I32, I64, I64, I64, I32, P, P, P, P, P, P, P]),
        "fp4_amax": (I32, [P, I32, I64, I64, I64, P, P]),
        "fp4_dequantize": (I32, [P, I64, I64, P, I32, P]),
        "fp4_gemm": (I32, [P, P, P, I32, I64, I64, I64, P]),
        "fp4q_linear_workspace_size": (SZ, [I32, I64, I64, I64]),
        "fp4_linear": (I32, [P, I32, I64, P, I64, I64, I64, P, P, I32, P, SZ, P]),
        "fp4q_linear_train_workspace_size": (SZ, [I32, I64, I64, I64]),
        "fp4_linear_train": (I32, [P, P, P, I32, I64, I64, I64, I32, P, P, P, I32, P, SZ, P]),
        "fp8_act_forward": (I32, [I32, I32, I64, I64, P, I64, P, I64, P, I64, P, P, P, P, P]),
        "fp8_act_backward": (I32, [I32, I32, I64, I64, P, P, P, P, P, I64, P, I64, P, I64, P,
                                   I64, P]),
        "fp8_rmsnorm": (I32, [P, I64, P, I64, I32, P, I32, P, I64, I64, P, I64, P, I64, I32, P, P,
                              P, P]),
        "fp8q_rmsnorm_backward_workspace_size": (SZ, [I64, I64]),
        "fp8_rmsnorm_backward": (I32, [P, I64, P, I64, I32, P, I32, P, P, I64, I64, I64, P, I64, P,
                                       P, SZ, P]),
        "fp8q_experts_blocks": (I64, [I64, I32, I32]),
        "fp8q_experts_scale_bytes": (SZ, [I64, I64, I32, I32]),
        "fp8_quantize_experts": (I32, [P, I32, I64, I64, P, P, P]),
        "fp8_experts_fprop": (I32, [P, P, P, I32, P]),
        "fp8_experts_dgrad": (I32, [P, P, P, I32, P]),
        "fp8_experts_wgrad": (I32, [P, P, P, I32, P]),
    }


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfp8q.so (built by ``build_lib``); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} not found: build it with `python -m scaled_quantize_fp8_warp_gb300.build_lib`"
                " (the FP8 path has no fallback)")
        lib = ctypes.CDLL(path)
        sig = signatures()
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def lib() -> ctypes.CDLL:
    return _lib if _lib is not None else load_library()


# --------------------------------------------------------------- marshalling

def _check(status: int, what: str):
    if status != OK:
        raise Fp8qError(status, what)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fp8q needs CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("fp8q needs contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _in_dtype(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return DT_BF16
    if x.dtype == torch.float32:
        return DT_F32
    raise TypeError(f"input must be bfloat16 or float32, got {x.dtype}")


_DT = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}


def _out_dtype(dt) -> int:
    if dt == torch.bfloat16:
        return DT_BF16
    if dt == torch.float32:
        return DT_F32
    raise TypeError(f"output must be bfloat16 or float32, got {dt}")


def _rows_cols(x: torch.Tensor):
    if x.dim() != 2:
        raise ValueError("expected a 2-D matrix")
    return x.shape[0], x.shape[1]


def _empty(shape, dtype, like: torch.Tensor):
    return torch.empty(shape, dtype=dtype, device=like.device)


# ------------------------------------------------------------------ a1 amax

def fp8_amax(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """max |x| into a 1-element fp32 device tensor."""
    out = out if out is not None else _empty((1,), torch.float32, x)
    _check(lib().fp8_amax(_ptr(x), _in_dtype(x), x.numel(), _ptr(out), _stream(stream)),
           "fp8_amax")
    return out


# --------------------------------------------------------- a2/a3 quantize

def fp8_quantize_tensor(x, fmt, amax, want_q=True, want_qt=False, saturate=False,
                        q=None, q_t=None, scale=None, stream=None):
    """Per-tensor current scaling with s from the device scalar ``amax``.
    Returns (q [R,C] uint8 | None, q_t [C,R] uint8 | None, scale [1] fp32)."""
    R, C = _rows_cols(x)
    if want_q and q is None:
        q = _empty((R, C), torch.uint8, x)
    if want_qt and q_t is None:
        q_t = _empty((C, R), torch.uint8, x)
    scale = scale if scale is not None else _empty((1,), torch.float32, x)
    _check(lib().fp8_quantize_tensor(_ptr(x), _in_dtype(x), R, C, fmt, _ptr(amax), _ptr(scale),
                                     _ptr(q if want_q else None), _ptr(q_t if want_qt else None),
                                     int(saturate), _stream(stream)), "fp8_quantize_tensor")
    return (q if want_q else None), (q_t if want_qt else None), scale


def fp8_quantize_tensor_current(x, fmt, want_q=True, want_qt=False, saturate=False, q=None,
                                q_t=None, amax=None, scale=None, stream=None):
    """amax and per-tensor cast in one call (one cooperative launch when x
    holds at most 8 MiB).  Returns (q | None, q_t | None, amax [1], scale [1])."""
    R, C = _rows_cols(x)
    if want_q and q is None:
        q = _empty((R, C), torch.uint8, x)
    if want_qt and q_t is None:
        q_t = _empty((C, R), torch.uint8, x)
    amax = amax if amax is not None else _empty((1,), torch.float32, x)
    scale = scale if scale is not None else _empty((1,), torch.float32, x)
    _check(lib().fp8_quantize_tensor_current(
        _ptr(x), _in_dtype(x), R, C, fmt, _ptr(amax), _ptr(scale), _ptr(q if want_q else None),
        _ptr(q_t if want_qt else None), int(saturate), _stream(stream)),
        "fp8_quantize_tensor_current")
    return (q if want_q else None), (q_t if want_qt else None), amax, scale


class History:
    """Device-resident delayed-scaling state (fp8q_amax_history, 80 bytes)."""

    def __init__(self, device=None, initial=None, stream=None):
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.buf = torch.empty(HISTORY_BYTES // 4, dtype=torch.int32, device=dev)
        self.reset(initial, stream)

    def reset(self, initial=None, stream=None):
        arr = None
        if initial is not None:
            vals = [float(v) for v in initial]
            if len(vals) != HISTORY_LEN:
                raise ValueError(f"history needs {HISTORY_LEN} values")
            arr = (ctypes.c_float * HISTORY_LEN)(*vals)
        _check(lib().fp8q_history_init(_ptr(self.buf), arr, _stream(stream)), "fp8q_history_init")

    def state(self):
        """(amax list, next, scale) read back to the host (synchronises)."""
        h = self.buf.cpu()
        f = h.view(torch.float32)
        return f[:HISTORY_LEN].tolist(), int(h[HISTORY_LEN]), float(f[HISTORY_LEN + 1])

    def scratch(self):
        h = self.buf.cpu()
        return int(h[HISTORY_LEN + 2]), int(h[HISTORY_LEN + 3])


def fp8_quantize_delayed(x, fmt, hist: History, want_q=True, want_qt=False, saturate=False,
                         q=None, q_t=None, scale=None, stream=None):
    R, C = _rows_cols(x)
    if want_q and q is None:
        q = _empty((R, C), torch.uint8, x)
    if want_qt and q_t is None:
        q_t = _empty((C, R), torch.uint8, x)
    scale = scale if scale is not None else _empty((1,), torch.float32, x)
    _check(lib().fp8_quantize_delayed(_ptr(x), _in_dtype(x), R, C, fmt, _ptr(hist.buf),
                                      _ptr(scale), _ptr(q if want_q else None),
                                      _ptr(q_t if want_qt else None), int(saturate),
                                      _stream(stream)), "fp8_quantize_delayed")
    return (q if want_q else None), (q_t if want_qt else None), scale


def fp8_quantize_tile1x128(x, fmt, rows=True, cols=False, saturate=False, q=None,
                           q_scales=None, q_t=None, qt_scales=None, stream=None):
    """1x128 row tiles (q [R,C], q_scales [ceil(C/128), R]) and/or 128x1 column
    tiles (q_t [C,R], qt_scales [ceil(R/128), C]) from one read of x."""
    R, C = _rows_cols(x)
    if rows:
        q = q if q is not None else _empty((R, C), torch.uint8, x)
        q_scales = q_scales if q_scales is not None else _empty(((C + 127) // 128, R),
                                                                torch.float32, x)
    if cols:
        q_t = q_t if q_t is not None else _empty((C, R), torch.uint8, x)
        qt_scales = qt_scales if qt_scales is not None else _empty(((R + 127) // 128, C),
                                                                   torch.float32, x)
    _check(lib().fp8_quantize_tile1x128(
        _ptr(x), _in_dtype(x), R, C, fmt, _ptr(q if rows else None),
        _ptr(q_scales if rows else None), _ptr(q_t if cols else None),
        _ptr(qt_scales if cols else None), int(saturate), _stream(stream)),
        "fp8_quantize_tile1x128")
    return ((q, q_scales) if rows else (None, None)) + ((q_t, qt_scales) if cols else (None, None))


def fp8_quantize_rowwise(x, fmt, rows=True, cols=False, saturate=False, q=None, q_scales=None,
                         q_t=None, qt_scales=None, stream=None):
    """Row-wise scaling: q [R,C] with q_scales [R] (one scale per row) and/or
    q_t [C,R] with qt_scales [C] (one scale per column of x)."""
    R, C = _rows_cols(x)
    if rows:
        q = q if q is not None else _empty((R, C), torch.uint8, x)
        q_scales = q_scales if q_scales is not None else _empty((R,), torch.float32, x)
    if cols:
        q_t = q_t if q_t is not None else _empty((C, R), torch.uint8, x)
        qt_scales = qt_scales if qt_scales is not None else _empty((C,), torch.float32, x)
    _check(lib().fp8_quantize_rowwise(
        _ptr(x), _in_dtype(x), R, C, fmt, _ptr(q if rows else None),
        _ptr(q_scales if rows else None), _ptr(q_t if cols else None),
        _ptr(qt_scales if cols else None), int(saturate), _stream(stream)),
        "fp8_quantize_rowwise")
    return ((q, q_scales) if rows else (None, None)) + ((q_t, qt_scales) if cols else (None, None))


def mx_scale_bytes(rows: int, cols: int) -> int:
    """Bytes of one orientation's MXFP8 scale atoms for an [rows, cols] matrix."""
    return int(lib().fp8q_mx_scale_bytes(rows, cols))


def fp8_quantize_mxfp8(x, fmt, rows=True, cols=False, q=None, q_scales=None, q_t=None,
                       qt_scales=None, stream=None):
    """MXFP8 (OCP MX v1.0): q [R,C] with 1x32 row blocks and/or q_t [C,R] with
    32x1 column blocks of x; scales are E8M0 bytes in the library's atom
    layout (uint8 tensors of mx_scale_bytes(R, C) bytes; see include/fp8q.h).
    Returns (q, q_scales, q_t, qt_scales), None for a pair not requested."""
    R, C = _rows_cols(x)
    nbytes = mx_scale_bytes(R, C)
    if rows:
        q = q if q is not None else _empty((R, C), torch.uint8, x)
        q_scales = q_scales if q_scales is not None else _empty((nbytes,), torch.uint8, x)
    if cols:
        q_t = q_t if q_t is not None else _empty((C, R), torch.uint8, x)
        qt_scales = qt_scales if qt_scales is not None else _empty((nbytes,), torch.uint8, x)
    _check(lib().fp8_quantize_mxfp8(
        _ptr(x), _in_dtype(x), R, C, fmt, _ptr(q if rows else None),
        _ptr(q_scales if rows else None), _ptr(q_t if cols else None),
        _ptr(qt_scales if cols else None), _stream(stream)), "fp8_quantize_mxfp8")
    return ((q, q_scales) if rows else (None, None)) + ((q_t, qt_scales) if cols else (None, None))


def fp8_quantize_block128x128(x, fmt, want_q=True, want_qt=False, saturate=False, q=None,
                              q_t=None, scales=None, stream=None):
    R, C = _rows_cols(x)
    if want_q and q is None:
        q = _empty((R, C), torch.uint8, x)
    if want_qt and q_t is None:
        q_t = _empty((C, R), torch.uint8, x)
    scales = scales if scales is not None else _empty(((R + 127) // 128, (C + 127) // 128),
                                                      torch.float32, x)
    _check(lib().fp8_quantize_block128x128(_ptr(x), _in_dtype(x), R, C, fmt,
                                           _ptr(q if want_q else None),
                                           _ptr(q_t if want_qt else None), _ptr(scales),
                                           int(saturate), _stream(stream)),
           "fp8_quantize_block128x128")
    return (q if want_q else None), (q_t if want_qt else None), scales


# ------------------------------------------------------------- a4/a5 GEMM

class GemmOperand:
    """An FP8 operand [rows, K] (uint8 device tensor) with its scales; keeps
    the tensors alive next to the ctypes struct."""

    def __init__(self, data: torch.Tensor, fmt: int, scaling: int, scale: torch.Tensor,
                 stride_row: int = 0, stride_k: int = 0):
        if data.dtype != torch.uint8 or data.dim() != 2:
            raise TypeError("operand data must be a 2-D uint8 tensor")
        self.data, self.scale = data, scale
        self.rows, self.K = data.shape
        self.struct = Operand(data.data_ptr(), fmt, scaling, scale.data_ptr(), stride_row,
                              stride_k)

    @classmethod
    def tensor(cls, q, fmt, scale):
        return cls(q, fmt, SCALE_TENSOR, scale)

    @classmethod
    def tile(cls, q, fmt, scales):
        """scales [ceil(K/128), rows] as written by fp8_quantize_tile1x128."""
        return cls(q, fmt, SCALE_TILE_1x128, scales, 1, q.shape[0])

    @classmethod
    def row(cls, q, fmt, scales):
        """One scale per row over all of K (scales [rows])."""
        return cls(q, fmt, SCALE_ROW, scales, 1, 0)

    @classmethod
    def mx(cls, q, fmt, atoms):
        """MXFP8 operand: atoms as fp8_quantize_mxfp8 writes them for q."""
        return cls(q, fmt, SCALE_MX_1x32, atoms, 0, 0)

    @classmethod
    def block(cls, q, fmt, scales):
        """scales [ceil(rows/128), ceil(K/128)] of this orientation."""
        return cls(q, fmt, SCALE_BLOCK_128x128, scales, scales.shape[1], 1)

    @classmethod
    def block_transposed(cls, q_t, fmt, scales):
        """q_t = q^T of a block-quantised matrix; scales as written for q."""
        return cls(q_t, fmt, SCALE_BLOCK_128x128, scales, 1, scales.shape[1])


class GemmDesc(ctypes.Structure):
    """fp8q_gemm_desc: one GEMM of an fp8_gemm_grouped call."""
    _fields_ = [("A", Operand), ("B", Operand), ("C", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


#: most GEMMs one fp8_gemm_grouped call takes (FP8Q_GEMM_GROUP_MAX)
GEMM_GROUP_MAX = 3


def fp8_gemm_grouped(problems, out_dtype=torch.bfloat16, outs=None, stream=None):
    """Up to three independent GEMMs in one call: problems = [(A, B), ...]
    with C_i = A_i . B_i^T as fp8_gemm computes it (one launch when the
    CTA-pair kernel runs them all).  Returns the outputs."""
    problems = list(problems)
    outs = list(outs) if outs is not None else [
        torch.empty((A.rows, B.rows), dtype=out_dtype, device=A.data.device) for A, B in problems]
    if len(outs) != len(problems):
        raise ValueError("one output per problem")
    arr = (GemmDesc * max(1, len(problems)))()
    for i, ((A, B), C) in enumerate(zip(problems, outs)):
        arr[i] = GemmDesc(A.struct, B.struct, _ptr(C), A.rows, B.rows, A.K)
    dt = _out_dtype(outs[0].dtype) if outs else _out_dtype(out_dtype)
    _check(lib().fp8_gemm_grouped(ctypes.cast(arr, ctypes.c_void_p), len(problems), dt,
                                  _stream(stream)), "fp8_gemm_grouped")
    return outs


def _gemm_call(fn_name, A: GemmOperand, B: GemmOperand, out, M, N, K, stream):
    fn = getattr(lib(), fn_name)
    _check(fn(ctypes.byref(A.struct), ctypes.byref(B.struct), _ptr(out), _out_dtype(out.dtype),
              M, N, K, _stream(stream)), fn_name)
    return out


def fp8_gemm(A: GemmOperand, B: GemmOperand, out_dtype=torch.bfloat16, out=None, stream=None):
    """C [M, N] = A [M, K] . B [N, K]^T, dequantised."""
    M, N = A.rows, B.rows
    out = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=A.data.device)
    return _gemm_call("fp8_gemm", A, B, out, M, N, A.K, stream)


def fp8_gemm_amax(A: GemmOperand, B: GemmOperand, out_dtype=torch.bfloat16, out=None,
                  amax=None, stream=None):
    """fp8_gemm plus amax(|C|) over the stored output from the same launch.
    Returns (C, amax) with amax a one-element fp32 device tensor."""
    M, N = A.rows, B.rows
    out = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=A.data.device)
    amax = amax if amax is not None else _empty((1,), torch.float32, A.data)
    _check(lib().fp8_gemm_amax(ctypes.byref(A.struct), ctypes.byref(B.struct), _ptr(out),
                               _out_dtype(out.dtype), M, N, A.K, _ptr(amax), _stream(stream)),
           "fp8_gemm_amax")
    return out, amax


def fp8_gemm_fprop(x: GemmOperand, w: GemmOperand, out_dtype=torch.bfloat16, out=None,
                   stream=None):
    M, K, N = x.rows, x.K, w.rows
    out = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=x.data.device)
    return _gemm_call("fp8_gemm_fprop", x, w, out, M, N, K, stream)


def fp8_gemm_dgrad(g: GemmOperand, w_t: GemmOperand, out_dtype=torch.bfloat16, out=None,
                   stream=None):
    M, N, K = g.rows, g.K, w_t.rows
    out = out if out is not None else torch.empty((M, K), dtype=out_dtype, device=g.data.device)
    return _gemm_call("fp8_gemm_dgrad", g, w_t, out, M, N, K, stream)


def fp8_gemm_wgrad(g_t: GemmOperand, x_t: GemmOperand, out_dtype=torch.bfloat16, out=None,
                   stream=None):
    N, M, K = g_t.rows, g_t.K, x_t.rows
    out = out if out is not None else torch.empty((N, K), dtype=out_dtype, device=g_t.data.device)
    return _gemm_call("fp8_gemm_wgrad", g_t, x_t, out, M, N, K, stream)


# ------------------------------------------------------------ whole forward

def linear_workspace_size(recipe: int, M: int, N: int, K: int) -> int:
    return int(lib().fp8q_linear_workspace_size(recipe, M, N, K))


def fp8_linear_autocast(x, w, recipe=RECIPE_TENSOR_CURRENT, out_dtype=torch.bfloat16,
                        hist_x: History | None = None, hist_w: History | None = None,
                        workspace=None, out=None, stream=None):
    """y = x w^T with dynamic FP8 quantisation of x and w (autocast)."""
    M, K = _rows_cols(x)
    N = w.shape[0]
    need = linear_workspace_size(recipe, M, N, K)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    out = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check(lib().fp8_linear_autocast(
        _ptr(x), _ptr(w), _in_dtype(x), M, N, K, recipe,
        _ptr(hist_x.buf) if hist_x else None, _ptr(hist_w.buf) if hist_w else None,
        _ptr(out), _out_dtype(out.dtype), _ptr(workspace), workspace.numel(), _stream(stream)),
        "fp8_linear_autocast")
    return out


def linear_train_workspace_size(recipe: int, M: int, N: int, K: int) -> int:
    return int(lib().fp8q_linear_train_workspace_size(recipe, M, N, K))


def fp8_linear_train(x, w, g, recipe=RECIPE_TENSOR_CURRENT, out_dtype=torch.bfloat16,
                     hist_x: History | None = None, hist_w: History | None = None,
                     hist_g: History | None = None, workspace=None, y=None, dx=None, dw=None,
                     stream=None):
    """One linear layer's Fprop, Dgrad and Wgrad with x, w, grad_out quantized
    on the fly (device tensors).  Returns (y, dx, dw)."""
    M, K = _rows_cols(x)
    N = w.shape[0]
    if workspace is None:
        workspace = torch.empty(linear_train_workspace_size(recipe, M, N, K), dtype=torch.uint8,
                                device=x.device)
    y = y if y is not None else torch.empty((M, N), dtype=out_dtype, device=x.device)
    dx = dx if dx is not None else torch.empty((M, K), dtype=out_dtype, device=x.device)
    dw = dw if dw is not None else torch.empty((N, K), dtype=out_dtype, device=x.device)
    hp = lambda h: _ptr(h.buf) if h else None
    _check(lib().fp8_linear_train(
        _ptr(x), _ptr(w), _ptr(g), _in_dtype(x), M, N, K, recipe, hp(hist_x), hp(hist_w),
        hp(hist_g), _ptr(y), _ptr(dx), _ptr(dw), _out_dtype(y.dtype), _ptr(workspace),
        workspace.numel(), _stream(stream)), "fp8_linear_train")
    return y, dx, dw


def linear_train_host_workspace_size(recipe: int, in_dtype, out_dtype, M: int, N: int,
                                     K: int) -> int:
    return int(lib().fp8q_linear_train_host_workspace_size(
        recipe, _DT[in_dtype], _DT[out_dtype], M, N, K))


def fp8_linear_train_host(x_h, w_h, g_h, y_h, dx_h, dw_h, workspace,
                          recipe=RECIPE_TENSOR_CURRENT, hist_x: History | None = None,
                          hist_w: History | None = None, hist_g: History | None = None,
                          stream=None):
    """fp8_linear_train from and to host tensors (pinned CPU tensors; the
    copies happen inside the call's work on `stream`).  Outputs are filled
    once `stream` has reached this call's end."""
    M, K = x_h.shape
    N = w_h.shape[0]
    for t in (x_h, w_h, g_h, y_h, dx_h, dw_h):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host buffers must be contiguous CPU tensors")
    hp = lambda h: _ptr(h.buf) if h else None
    _check(lib().fp8_linear_train_host(
        x_h.data_ptr(), w_h.data_ptr(), g_h.data_ptr(), _DT[x_h.dtype], M, N, K, recipe,
        hp(hist_x), hp(hist_w), hp(hist_g), y_h.data_ptr(), dx_h.data_ptr(), dw_h.data_ptr(),
        _DT[y_h.dtype], _ptr(workspace), workspace.numel(), _stream(stream)),
        "fp8_linear_train_host")


#: size of the library's static scratch (FP8Q_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def fp8_linear_autocast_noalloc(x, w, recipe=RECIPE_TENSOR_CURRENT, out_dtype=torch.bfloat16,
                                hist_x: History | None = None, hist_w: History | None = None,
                                out=None, stream=None):
    """fp8_linear_autocast for callers that cannot allocate device memory:
    the library keeps the FP8 copies and scales in its own fixed 64 MiB
    device array (see include/fp8q.h), so only the output is supplied here.
    Pass ``out`` to make the call allocate nothing at all from Python either."""
    M, K = _rows_cols(x)
    N = w.shape[0]
    out = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check(lib().fp8_linear_autocast_noalloc(
        _ptr(x), _ptr(w), _in_dtype(x), M, N, K, recipe,
        _ptr(hist_x.buf) if hist_x else None, _ptr(hist_w.buf) if hist_w else None,
        _ptr(out), _out_dtype(out.dtype), _stream(stream)), "fp8_linear_autocast_noalloc")
    return out


# ------------------------------------------------------------ 4-bit formats

class _Fp4Struct(ctypes.Structure):
    """fp4q_operand."""
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("global_scale", ctypes.c_void_p), ("kind", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def _rows(t: torch.Tensor):
    """(pointer, row stride in elements) of a 2-D matrix whose rows are dense;
    the rows may lie apart (a slice of a wider matrix)."""
    if not t.is_cuda:
        raise ValueError("fp8q needs CUDA tensors")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("expected a 2-D matrix")
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    rows, cols = shape
    ld = t.stride(0) if rows > 1 else max(cols, 1)
    if (cols > 1 and t.stride(1) != 1) or ld < cols:
        raise ValueError("fp8q needs matrices whose rows are dense and do not overlap")
    return t.data_ptr(), ld


def _addr(t: torch.Tensor | None):
    """Pointer of a dense tensor."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fp8q needs CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("fp8q needs contiguous tensors")
    return t.data_ptr()


def _raw_stream(stream=None) -> int:
    """The CUDA stream's handle.  The raw query of the current one costs a
    thirtieth of building a Stream object (0.1 against 3 us on a Grace core)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _new(shape, dtype, device, stream):
    """Storage a call writes on ``stream``: allocated there, so that the
    caching allocator orders its reuse after that stream's work."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(t: torch.Tensor, shape, dtype, what: str):
    """Checks a caller's tensor against what a call is about to write or read."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of shape "
                         f"{tuple(t.shape)}")
    return t


def _one(t: torch.Tensor, what: str):
    """Pointer of a one-element fp32 device tensor."""
    if t.numel() != 1 or t.dtype != torch.float32:
        raise ValueError(f"{what} is one fp32 value")
    return _addr(t)


def _out(out, shape, dtype, device, stream, what="out"):
    """(tensor, its address, dtype code) of a dense result: the caller's,
    checked, or a new one."""
    if out is None:
        out = _new(shape, dtype, device, stream)
        return out, out.data_ptr(), _out_dtype(dtype)
    return _like(out, shape, out.dtype, what), _addr(out), _out_dtype(out.dtype)


def _out_rows(out, shape, dtype, device, stream, what):
    """(tensor, address, row stride) of a result whose rows may lie apart: the
    caller's, checked, or a new one."""
    if out is None:
        out = _new(shape, dtype, device, stream)
        return out, out.data_ptr(), shape[1]
    return _like(out, shape, dtype, what), *_rows(out)


def _given(t, shape, dtype, device, stream, what):
    """(tensor, its address) of a dense result of one type: the caller's,
    checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device) if stream is None else _new(
            shape, dtype, device, stream)
        return t, t.data_ptr()
    return t, _addr(_like(t, shape, dtype, what))


def _here(*tensors):
    """Refuses tensors of another device than the current one, on which a call
    runs (CUDA tensors or None)."""
    device = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("fp8q needs tensors on the current device")


def fp4_scale_bytes(kind: int, rows: int, K: int) -> int:
    """Bytes of the scale atoms of an [rows, K] 4-bit operand."""
    return (rows + 127) // 128 * ((K + 127) // 128 if kind == MXFP4 else (K + 63) // 64) * 512


class Fp4Operand:
    """A 4-bit operand [rows, K] (MXFP4 or NVFP4): packed codes [rows, 16
    ceil(K/32)] and scale atoms, both uint8 device tensors, and for NVFP4 the
    one-element fp32 tensor scale; see fp4q_operand in include/fp8q.h."""
    __slots__ = ("data", "scales", "kind", "rows", "K", "global_scale", "struct")

    def __init__(self, data: torch.Tensor, scales: torch.Tensor, kind: int, K: int,
                 global_scale: torch.Tensor | None = None):
        if data.dim() != 2 or data.dtype != torch.uint8 or data.shape[1] != (K + 31) // 32 * 16:
            raise ValueError("4-bit data must be uint8 [rows, 16 ceil(K/32)]")
        if kind not in (MXFP4, NVFP4):
            raise ValueError("a 4-bit operand is MXFP4 or NVFP4")
        rows = data.shape[0]
        need = fp4_scale_bytes(kind, rows, K)
        if scales.dtype != torch.uint8 or scales.numel() != need:
            raise ValueError(f"4-bit scales must be {need} uint8 values")
        if (kind == NVFP4) != (global_scale is not None):
            raise ValueError("NVFP4 operands, and only they, have a global scale")
        g = None if global_scale is None else _one(global_scale, "a global scale")
        self.data, self.scales, self.kind, self.rows, self.K = data, scales, kind, rows, K
        self.global_scale = global_scale
        self.struct = _Fp4Struct(_addr(data), _addr(scales), g, kind, 0)

    @classmethod
    def empty(cls, kind: int, rows: int, K: int, device, global_scale=None, stream=None):
        """Uninitialised storage for an operand."""
        op = cls.__new__(cls)
        op.data = data = _new((rows, (K + 31) // 32 * 16), torch.uint8, device, stream)
        op.scales = scales = _new((fp4_scale_bytes(kind, rows, K),), torch.uint8, device, stream)
        op.kind, op.rows, op.K, op.global_scale = kind, rows, K, global_scale
        g = None if global_scale is None else _one(global_scale, "a global scale")
        op.struct = _Fp4Struct(data.data_ptr(), scales.data_ptr(), g, kind, 0)
        return op


def fp4_amax(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """max |x| of a matrix whose rows may lie apart, as a one-element fp32 tensor."""
    p, ld = _rows(x)
    out = out if out is not None else _new((1,), torch.float32, x.device, stream)
    _check(lib().fp4_amax(p, _in_dtype(x), x.shape[0], x.shape[1], ld, _one(out, "out"),
                          _raw_stream(stream)), "fp4_amax")
    return out


def fp4_quantize(x: torch.Tensor, kind: int, rows=True, cols=False,
                 amax: torch.Tensor | None = None, q: Fp4Operand | None = None,
                 q_t: Fp4Operand | None = None, stream=None):
    """x [R, C] (rows may lie apart) -> (operand [R, C] | None, operand [C, R]
    of x^T | None).  NVFP4 takes the tensor's amax from ``amax`` (one fp32
    device value) or finds it first.  ``q`` and ``q_t`` are storage for the
    orientations asked for by ``rows`` and ``cols``, which share one tensor
    scale; one that is not asked for is not touched."""
    p, ld = _rows(x)
    R, C = x.shape
    if kind not in (MXFP4, NVFP4):
        raise ValueError("a 4-bit operand is MXFP4 or NVFP4")
    q, q_t, g = (q if rows else None), (q_t if cols else None), None
    if kind == NVFP4:
        amax = amax if amax is not None else fp4_amax(x, stream=stream)
        given = q if q is not None else q_t
        g = given.global_scale if given is not None else _new((1,), torch.float32, x.device, stream)
    if rows:
        q = q if q is not None else Fp4Operand.empty(kind, R, C, x.device, g, stream)
        if (q.kind, q.rows, q.K) != (kind, R, C):
            raise ValueError(f"an operand of kind, rows, K {(kind, R, C)} is needed")
    if cols:
        q_t = q_t if q_t is not None else Fp4Operand.empty(kind, C, R, x.device, g, stream)
        if (q_t.kind, q_t.rows, q_t.K) != (kind, C, R):
            raise ValueError(f"an operand of kind, rows, K {(kind, C, R)} is needed")
    if rows and cols and kind == NVFP4 and q.global_scale.data_ptr() != q_t.global_scale.data_ptr():
        raise ValueError("both orientations share one global scale")
    a, b = (q.struct if rows else None), (q_t.struct if cols else None)
    _check(lib().fp4_quantize(
        p, _in_dtype(x), R, C, ld, kind, _one(amax, "amax") if kind == NVFP4 else None,
        a.data if rows else None, a.scales if rows else None, b.data if cols else None,
        b.scales if cols else None, _addr(g), _raw_stream(stream)), "fp4_quantize")
    return q, q_t


def fp4_dequantize(op: Fp4Operand, out_dtype=torch.bfloat16, out=None, stream=None):
    """The values [rows, K] an operand stands for."""
    out, po, dt = _out(out, (op.rows, op.K), out_dtype, op.data.device, stream)
    _check(lib().fp4_dequantize(ctypes.byref(op.struct), op.rows, op.K, po, dt,
                                _raw_stream(stream)), "fp4_dequantize")
    return out


def fp4_gemm(A: Fp4Operand, B: Fp4Operand, out_dtype=torch.bfloat16, out=None, stream=None):
    """C [M, N] = A [M, K] . B [N, K]^T of two operands of one kind."""
    if A.K != B.K:
        raise ValueError(f"operands contract over {A.K} and {B.K}")
    out, po, dt = _out(out, (A.rows, B.rows), out_dtype, A.data.device, stream)
    _check(lib().fp4_gemm(ctypes.byref(A.struct), ctypes.byref(B.struct), po, dt, A.rows,
                          B.rows, A.K, _raw_stream(stream)), "fp4_gemm")
    return out


def fp4_linear_workspace_size(kind: int, M: int, N: int, K: int) -> int:
    return int(lib().fp4q_linear_workspace_size(kind, M, N, K))


#: most rows of x that fp4_linear quantises inside the product (FP4Q_LINEAR_FUSED_ROWS)
FP4_LINEAR_FUSED_ROWS = 16


def fp4_linear(x: torch.Tensor, w: Fp4Operand, x_amax: torch.Tensor | None = None,
               out_dtype=torch.bfloat16, workspace=None, out=None, stream=None):
    """y [M, N] = x w^T with w [N, K] held in 4 bits: x [M, K] (rows may lie
    apart) is quantised to w's kind in the call.  ``x_amax``: a calibrated
    amax of x for NVFP4 (one fp32 device value); without it the call finds
    max |x|."""
    p, ld = _rows(x)
    M, K = x.shape
    N, kind = w.rows, w.kind
    if K != w.K:
        raise ValueError(f"x has {K} columns, w contracts over {w.K}")
    if workspace is None and not (M <= FP4_LINEAR_FUSED_ROWS
                                  and (kind == MXFP4 or x_amax is not None)):
        workspace = _new((fp4_linear_workspace_size(kind, M, N, K),), torch.uint8, x.device, stream)
    out, po, dt = _out(out, (M, N), out_dtype, x.device, stream)
    _check(lib().fp4_linear(
        p, _in_dtype(x), ld, ctypes.byref(w.struct), M, N, K,
        None if x_amax is None else _one(x_amax, "x_amax"), po, dt, _addr(workspace),
        0 if workspace is None else workspace.numel(), _raw_stream(stream)), "fp4_linear")
    return out


def fp4_linear_train_workspace_size(kind: int, M: int, N: int, K: int) -> int:
    return int(lib().fp4q_linear_train_workspace_size(kind, M, N, K))


def fp4_linear_train(x, w, g, kind: int, out_dtype=torch.bfloat16, workspace=None, y=None,
                     dx=None, dw=None, stream=None):
    """One linear layer's Fprop, Dgrad and Wgrad in 4 bits, every operand
    quantised in the call (device tensors).  Returns (y, dx, dw)."""
    M, K = _rows_cols(x)
    N = w.shape[0]
    _like(w, (N, K), x.dtype, "w")
    _like(g, (M, N), x.dtype, "g")
    if workspace is None:
        workspace = _new((fp4_linear_train_workspace_size(kind, M, N, K),), torch.uint8, x.device,
                         stream)
    y, py, dt = _out(y, (M, N), out_dtype, x.device, stream, "y")
    dx, pdx, _ = _out(dx, (M, K), y.dtype, x.device, stream, "dx")
    dw, pdw, _ = _out(dw, (N, K), y.dtype, x.device, stream, "dw")
    if dx.dtype != y.dtype or dw.dtype != y.dtype:
        raise ValueError("y, dx and dw have one type")
    _check(lib().fp4_linear_train(
        _addr(x), _addr(w), _addr(g), _in_dtype(x), M, N, K, kind, py, pdx, pdw, dt,
        _addr(workspace), workspace.numel(), _raw_stream(stream)), "fp4_linear_train")
    return y, dx, dw


# ------------------------------- activation functions with 8-bit checkpoints

class ActCheckpoint:
    """What fp8_act_forward keeps for the backward pass: E4M3 bytes [T, F]
    (uint8) of u, and of v for a gated activation, under 1x128 tile scales
    (fp32 [ceil(F/128), T])."""
    __slots__ = ("T", "F", "u", "u_scales", "v", "v_scales")

    def __init__(self, u: torch.Tensor, u_scales: torch.Tensor, v: torch.Tensor | None = None,
                 v_scales: torch.Tensor | None = None):
        self.T, self.F = _rows_cols(u)
        if (v is None) != (v_scales is None):
            raise ValueError("v and v_scales come together")
        shape = ((self.F + 127) // 128, self.T)
        _like(u, (self.T, self.F), torch.uint8, "checkpoint bytes")
        _like(u_scales, shape, torch.float32, "checkpoint scales")
        if v is not None:
            _like(v, (self.T, self.F), torch.uint8, "checkpoint bytes")
            _like(v_scales, shape, torch.float32, "checkpoint scales")
        self.u, self.u_scales, self.v, self.v_scales = u, u_scales, v, v_scales

    @classmethod
    def empty(cls, T: int, F: int, gated: bool, device, stream=None):
        """Uninitialised storage for a checkpoint."""
        c = cls.__new__(cls)
        c.T, c.F, shape = T, F, ((F + 127) // 128, T)
        c.u = _new((T, F), torch.uint8, device, stream)
        c.u_scales = _new(shape, torch.float32, device, stream)
        c.v = _new((T, F), torch.uint8, device, stream) if gated else None
        c.v_scales = _new(shape, torch.float32, device, stream) if gated else None
        return c


def fp8_act_forward(act: int, u: torch.Tensor, v: torch.Tensor | None = None, out=None,
                    ckpt: ActCheckpoint | None = None, stream=None):
    """(a, checkpoint) with a = f(u), or f(u) * v.  u and v are [T, F] of one
    type; their rows may lie apart (the two halves of one matrix)."""
    pu, ldu = _rows(u)
    T, F = u.shape
    pv, ldv = None, 0
    if v is not None:
        pv, ldv = _rows(_like(v, (T, F), u.dtype, "v"))
    out, pa, lda = _out_rows(out, (T, F), u.dtype, u.device, stream, "out")
    if ckpt is None:
        ckpt = ActCheckpoint.empty(T, F, v is not None, u.device, stream)
    elif (ckpt.T, ckpt.F, ckpt.v is None) != (T, F, v is None):
        raise ValueError("the checkpoint's shape is another")
    _check(lib().fp8_act_forward(
        act, _in_dtype(u), T, F, pu, ldu, pv, ldv, pa, lda, _addr(ckpt.u), _addr(ckpt.u_scales),
        _addr(ckpt.v), _addr(ckpt.v_scales), _raw_stream(stream)), "fp8_act_forward")
    return out, ckpt


def fp8_act_backward(act: int, ckpt: ActCheckpoint, da: torch.Tensor, want_a=False, du=None,
                     dv=None, a=None, stream=None):
    """(du, dv | None, a | None) from the checkpoint and the gradient of a;
    ``want_a`` (or a given ``a``) asks for the activation again."""
    shape, dtype, device = (ckpt.T, ckpt.F), da.dtype, da.device
    pd, ldd = _rows(_like(da, shape, dtype, "da"))
    if ckpt.v is None and dv is not None:
        raise ValueError("an ungated activation has no dv")
    du, pu, ldu = _out_rows(du, shape, dtype, device, stream, "du")
    pv, ldv, pa, lda = None, 0, None, 0
    if ckpt.v is not None:
        dv, pv, ldv = _out_rows(dv, shape, dtype, device, stream, "dv")
    if want_a or a is not None:
        a, pa, lda = _out_rows(a, shape, dtype, device, stream, "a")
    _check(lib().fp8_act_backward(
        act, _in_dtype(da), ckpt.T, ckpt.F, _addr(ckpt.u), _addr(ckpt.u_scales), _addr(ckpt.v),
        _addr(ckpt.v_scales), pd, ldd, pu, ldu, pv, ldv, pa, lda, _raw_stream(stream)),
        "fp8_act_backward")
    return du, dv, a


# ------------------------------------------- RMS norm with an 8-bit output

class NormOutput(NamedTuple):
    """What fp8_rmsnorm gives.  ``h`` [T, C]: x + residual as it is stored (x
    itself without a residual).  ``y`` [T, C] or None.  ``q`` [T, C] E4M3 bytes
    (uint8) with ``scales`` ([ceil(C/128), T] per tile, [T] per row), or None:
    an operand for GemmOperand.tile or GemmOperand.row.  ``rstd`` [T] fp32."""
    h: torch.Tensor
    y: torch.Tensor | None
    q: torch.Tensor | None
    scales: torch.Tensor | None
    rstd: torch.Tensor


def _norm_weight(weight: torch.Tensor, C: int):
    """(pointer, dtype code) of a norm's weight."""
    if weight.shape != (C,):
        raise ValueError(f"weight must have shape ({C},), got {tuple(weight.shape)}")
    return _addr(weight), _in_dtype(weight)


def fp8_rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                eps: float = 1e-6, scaling: int | None = SCALE_TILE_1x128, want_y=True, h=None,
                y=None, q=None, scales=None, rstd=None, stream=None) -> NormOutput:
    """h = x + residual, y = weight h / sqrt(mean(h^2) + eps), and y in E4M3 under
    1x128 tile scales or row scales (``scaling`` None: no 8-bit output).  x,
    residual, h and y are [T, C] of one type and their rows may lie apart;
    weight is bf16 or fp32.  ``want_y`` (or a given ``y``) asks for y beside
    its 8-bit form.  h may be x or residual itself; no other result overlaps an
    input."""
    px, ldx = _rows(x)
    T, C = shape = x.shape
    dtype, device = x.dtype, x.device
    pw, w_dtype = _norm_weight(weight, C)
    pr = ph = py = pq = ps = None
    ldr = ldh = ldy = 0
    if residual is not None:
        pr, ldr = _rows(_like(residual, shape, dtype, "residual"))
        if h is None:
            h, ph = _given(None, shape, dtype, device, stream, "h")
            ldh = C
        else:
            ph, ldh = _rows(_like(h, shape, dtype, "h"))
    elif h is not None:
        raise ValueError("without a residual h is x")
    if y is not None:
        py, ldy = _rows(_like(y, shape, dtype, "y"))
    elif want_y:
        y, py = _given(None, shape, dtype, device, stream, "y")
        ldy = C
    if scaling is not None:
        q, pq = _given(q, shape, torch.uint8, device, stream, "q")
        scales, ps = _given(scales, ((C + 127) // 128, T) if scaling == SCALE_TILE_1x128 else (T,),
                            torch.float32, device, stream, "scales")
    elif q is not None or scales is not None:
        raise ValueError("an 8-bit output needs a scaling")
    rstd, pd = _given(rstd, (T,), torch.float32, device, stream, "rstd")
    _here(x, weight, residual, h, y, q, scales, rstd)
    status = lib().fp8_rmsnorm(
        px, ldx, pr, ldr, _in_dtype(x), pw, w_dtype, ctypes.byref(ctypes.c_float(eps)), T, C, ph,
        ldh, py, ldy, scaling or 0, pq, ps, pd, _raw_stream(stream))
    if status != OK:
        raise Fp8qError(status, "fp8_rmsnorm")
    return NormOutput(x if h is None else h, y, q, scales, rstd)


def fp8_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                         rstd: torch.Tensor, dresidual: torch.Tensor | None = None,
                         want_dweight=True, dx=None, dweight=None, workspace=None, stream=None):
    """(dx, dweight | None) of fp8_rmsnorm from the gradient dy of y and the h
    and rstd that it gave; dx includes ``dresidual``, the gradient that reaches
    h by its other use."""
    pd, ldd = _rows(dy)
    T, C = shape = dy.shape
    dtype, device = dy.dtype, dy.device
    ph, ldh = _rows(_like(h, shape, dtype, "h"))
    pw, w_dtype = _norm_weight(weight, C)
    ps = _addr(_like(rstd, (T,), torch.float32, "rstd"))
    pr, ldr, pdw = None, 0, None
    if dresidual is not None:
        pr, ldr = _rows(_like(dresidual, shape, dtype, "dresidual"))
    dx, px, ldx = _out_rows(dx, shape, dtype, device, stream, "dx")
    if want_dweight or dweight is not None:
        dweight, pdw = _given(dweight, (C,), weight.dtype, device, stream, "dweight")
        if workspace is None:
            workspace = _new((lib().fp8q_rmsnorm_backward_workspace_size(T, C),), torch.uint8, device,
                             stream)
    _here(dy, h, weight, rstd, dresidual, dx, dweight, workspace)
    _check(lib().fp8_rmsnorm_backward(
        pd, ldd, ph, ldh, _in_dtype(dy), pw, w_dtype, ps, pr, ldr, T, C, px, ldx, pdw,
        _addr(workspace), 0 if workspace is None else workspace.numel(), _raw_stream(stream)),
        "fp8_rmsnorm_backward")
    return dx, dweight


# --------------------------------------- a linear layer per expert, in MXFP8

class _ExpertsStruct(ctypes.Structure):
    """fp8q_experts."""
    _fields_ = [("q", ctypes.c_void_p), ("q_scales", ctypes.c_void_p), ("q_t", ctypes.c_void_p),
                ("qt_scales", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("groups", ctypes.c_int32),
                ("format", ctypes.c_int32)]


#: most groups of an operand (FP8Q_EXPERTS_MAX)
EXPERTS_MAX = 1024


def experts_blocks(rows: int, groups: int, ragged: bool) -> int:
    """128-row blocks that the groups of an operand take."""
    return rows // 128 + groups if ragged else groups * ((rows // groups + 127) // 128)


class ExpertsOperand:
    """An MXFP8 operand [rows, cols] whose rows lie in groups, one per expert:
    group e has rows offsets[e] to offsets[e + 1] (``offsets``: int32 device
    tensor [groups + 1]), or rows / groups each where ``offsets`` is None (the
    weights of all experts, one below the other).  By rows: ``q`` uint8 [rows,
    cols] and ``q_scales``; transposed: ``q_t`` uint8 [cols, 128 blocks] and
    ``qt_scales``; scales are uint8, 512 * blocks * ceil(cols/128) of them.  See
    fp8q_experts in include/fp8q.h for where things lie.  An operand keeps the
    tensors it was made of: the calls use their addresses, found once; for other
    tensors (a step's new offsets over the same storage) make another operand."""
    __slots__ = ("_rows", "_cols", "_groups", "_fmt", "_offsets", "_q", "_q_scales", "_q_t",
                 "_qt_scales", "struct")
    rows, cols, groups, fmt, offsets, q, q_scales, q_t, qt_scales = (
        property(operator.attrgetter(name)) for name in __slots__[:-1])

    def __init__(self, rows: int, cols: int, groups: int, fmt: int = E4M3,
                 offsets: torch.Tensor | None = None, q: torch.Tensor | None = None,
                 q_scales: torch.Tensor | None = None, q_t: torch.Tensor | None = None,
                 qt_scales: torch.Tensor | None = None):
        if not 1 <= groups <= EXPERTS_MAX:
            raise ValueError(f"an operand has 1 to {EXPERTS_MAX} groups")
        if offsets is None:
            if rows % groups:
                raise ValueError("equal groups need rows that divide by their number")
        elif offsets.dtype != torch.int32 or offsets.shape != (groups + 1,):
            raise ValueError(f"offsets must be int32 of shape ({groups + 1},)")
        if (q is None) != (q_scales is None) or (q_t is None) != (qt_scales is None):
            raise ValueError("bytes and scales come together")
        blocks = experts_blocks(rows, groups, offsets is not None)
        for data, scales, shape in ((q, q_scales, (rows, cols)), (q_t, qt_scales, (cols, 128 * blocks))):
            if data is not None:
                _like(data, shape, torch.uint8, "bytes")
                if scales.dtype != torch.uint8 or scales.numel() != 512 * blocks * ((cols + 127) // 128):
                    raise ValueError(f"scales must be {512 * blocks * ((cols + 127) // 128)} uint8 values")
        self._rows, self._cols, self._groups, self._fmt, self._offsets = rows, cols, groups, fmt, offsets
        self._q, self._q_scales, self._q_t, self._qt_scales = q, q_scales, q_t, qt_scales
        self.struct = _ExpertsStruct(_addr(q), _addr(q_scales), _addr(q_t), _addr(qt_scales),
                                     _addr(offsets), rows, cols, groups, fmt)

    def tensors(self):
        """What the operand holds, None for what it lacks."""
        return self._q, self._q_scales, self._q_t, self._qt_scales, self._offsets

    @classmethod
    def empty(cls, rows: int, cols: int, groups: int, device, fmt: int = E4M3, offsets=None,
              by_rows=True, transposed=False, stream=None):
        """Uninitialised storage for an operand."""
        if not 1 <= groups <= EXPERTS_MAX:
            raise ValueError(f"an operand has 1 to {EXPERTS_MAX} groups")
        blocks = experts_blocks(rows, groups, offsets is not None)
        n = (512 * blocks * ((cols + 127) // 128),)
        q = qs = qt = qts = None
        if by_rows:
            q, qs = (_new(s, torch.uint8, device, stream) for s in ((rows, cols), n))
        if transposed:
            qt, qts = (_new(s, torch.uint8, device, stream) for s in ((cols, 128 * blocks), n))
        return cls(rows, cols, groups, fmt, offsets, q, qs, qt, qts)


def _same_offsets(a: torch.Tensor | None, b: torch.Tensor | None) -> bool:
    """Whether two sets of offsets are the same memory (or both equal groups)."""
    if a is None or b is None:
        return a is b
    return a is b or (a.data_ptr(), a.dtype, a.shape, a.stride()) == (b.data_ptr(), b.dtype, b.shape, b.stride())


def fp8_quantize_experts(x: torch.Tensor, groups: int, offsets: torch.Tensor | None = None,
                         index: torch.Tensor | None = None, rows=True, cols=False, fmt: int = E4M3,
                         out: ExpertsOperand | None = None, stream=None) -> ExpertsOperand:
    """x [T, C] (rows may lie apart) -> MXFP8 operand in groups, by rows, by
    columns (transposed) or both.  ``index`` (int32 device tensor): row r of the
    operand is row index[r] of x, a row of zeros where that is no row of x;
    without it row r is row r.  ``out``: storage, of which the orientations
    asked for are written."""
    p, ld = _rows(x)
    T, C = x.shape
    if index is not None and (index.dtype != torch.int32 or index.dim() != 1):
        raise ValueError("index must be int32, one for each row")
    S = T if index is None else index.shape[0]
    if not rows and not cols:
        raise ValueError("an orientation is needed: rows, cols or both")
    if out is None:
        out = ExpertsOperand.empty(S, C, groups, x.device, fmt, offsets, rows, cols, stream)
    elif (out.rows, out.cols, out.groups, out.fmt) != (S, C, groups, fmt) or not _same_offsets(
            out.offsets, offsets):
        raise ValueError("an operand of these rows, columns, groups, offsets and format is needed")
    st = out.struct
    if (rows and out.q is None) or (cols and out.q_t is None):
        raise ValueError("the operand has no storage for an orientation asked for")
    if (out.q is not None and not rows) or (out.q_t is not None and not cols):
        st = _ExpertsStruct(st.q if rows else None, st.q_scales if rows else None,
                            st.q_t if cols else None, st.qt_scales if cols else None, st.offsets,
                            S, C, groups, fmt)
    _here(x, index, *out.tensors())
    _check(lib().fp8_quantize_experts(p, _in_dtype(x), T, ld, _addr(index), ctypes.byref(st),
                                      _raw_stream(stream)), "fp8_quantize_experts")
    return out


def _experts_rows(name, x, w, shape, out_dtype, out, stream):
    held = x.q if x.q is not None else x.q_t
    if held is None:
        raise ValueError("an operand without bytes")
    device = held.device
    out, po, dt = _out(out, shape, out_dtype, device, stream)
    _here(out, *x.tensors(), *w.tensors())
    _check(getattr(lib(), name)(ctypes.byref(x.struct), ctypes.byref(w.struct), po, dt,
                                _raw_stream(stream)), name)
    return out


def fp8_experts_fprop(x: ExpertsOperand, w: ExpertsOperand, out_dtype=torch.bfloat16, out=None,
                      stream=None):
    """y [S, N], y_r = x_r w_e^T for rows r of group e, from x [S, K] by rows and
    the weights w [E N, K] by rows.  Rows of ``out`` behind the last group are
    left as they were (uninitialised in a new one)."""
    return _experts_rows("fp8_experts_fprop", x, w, (x.rows, w.rows // w.groups), out_dtype, out, stream)


def fp8_experts_dgrad(g: ExpertsOperand, w: ExpertsOperand, out_dtype=torch.bfloat16, out=None,
                      stream=None):
    """dx [S, K], dx_r = g_r w_e, from g [S, N] by rows and the weights w [E N, K]
    transposed.  Rows behind the last group as in fp8_experts_fprop."""
    return _experts_rows("fp8_experts_dgrad", g, w, (g.rows, w.cols), out_dtype, out, stream)


def fp8_experts_wgrad(g: ExpertsOperand, x: ExpertsOperand, out_dtype=torch.bfloat16, out=None,
                      stream=None):
    """dw [E, N, K], dw_e = g_e^T x_e, from g [S, N] and x [S, K] transposed, cast in
    the same groups; zero for an expert without rows.  Where the offsets of g and x are
    different tensors, dw_e is NaN for a group that is not the same rows in both."""
    return _experts_rows("fp8_experts_wgrad", g, x, (x.groups, g.cols, x.cols), out_dtype, out, stream)


# ------------------------------------------------------------- diagnostics

def device_status() -> int:
    """Synchronise and read (and clear) the device error word."""
    return int(lib().fp8q_device_status())


def selftest_barrier_timeout(stream=None) -> None:
    """Launch the failure-path self-test (see include/fp8q.h)."""
    _check(lib().fp8q_selftest_barrier_timeout(_stream(stream)), "fp8q_selftest_barrier_timeout")


def device_supported() -> bool:
    return bool(lib().fp8q_device_supported())


def status_string(status: int) -> str:
    return lib().fp8q_status_string(status).decode()
