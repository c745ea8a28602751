"""ctypes binding of libqlora (include/qlora.h), with the same entry-point names.

Argument marshalling only: tensors are PyTorch CUDA tensors (device memory and
streams), their data pointers and the current stream are passed to the C ABI,
and every step of the computation runs in the library's CUDA kernels.  There
is no CPU fallback: if ``lib/libqlora.so`` is missing, every call raises.

With the environment variable QLORA_LIBRARY=checked the binding loads the
bounds-checked debug build ``lib/libqlora_check.so`` instead (same ABI; its
kernels report an out-of-range index through the status word rather than
touching memory out of range).
"""

import ctypes
import math
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libqlora.so")
CHECK_LIB_PATH = os.path.join(_PKG, "lib", "libqlora_check.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "qlora.h")

QLORA_OK = 0
QLORA_ACT = {"swiglu": 0, "geglu_tanh": 1}
STATUS_NAMES = {0: "QLORA_OK", 1: "QLORA_ERR_INVALID_ARG", 2: "QLORA_ERR_UNSUPPORTED_SHAPE",
                3: "QLORA_ERR_MISALIGNED", 4: "QLORA_ERR_WORKSPACE_TOO_SMALL", 5: "QLORA_ERR_CUDA",
                6: "QLORA_ERR_TIMEOUT", 7: "QLORA_ERR_DEVICE"}


class QloraNF4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p),
                ("n_out", ctypes.c_int64), ("k_in", ctypes.c_int64)]


class QloraLoraLinear(ctypes.Structure):
    _fields_ = [("w", QloraNF4), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("r", ctypes.c_int32), ("scale", ctypes.c_float)]


class QloraLoraLinear16(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("n_out", ctypes.c_int64), ("k_in", ctypes.c_int64), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("r", ctypes.c_int32), ("scale", ctypes.c_float)]


class QloraFP8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("n_out", ctypes.c_int64), ("k_in", ctypes.c_int64)]


class QloraFP8Rows(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class QloraLoraLinear8(ctypes.Structure):
    _fields_ = [("w", QloraFP8), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("r", ctypes.c_int32), ("scale", ctypes.c_float)]


class QloraMlpSaved(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("E", "G", "H", "XA_g", "XA_u", "HA_d")]


class QloraTraceEntry(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


class QloraError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


_lib = None

_SIGS = {
    "qlora_nf4_codebook": (ctypes.c_int, [ctypes.c_void_p]),
    "nf4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p]),
    "nf4_dequantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_linear_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                       ctypes.c_int32]),
    "qlora_linear_fwd": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear), ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    "qlora_linear_bwd": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear), ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_mlp_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                    ctypes.c_int32]),
    "qlora_mlp_fwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(QloraLoraLinear),
                                     ctypes.POINTER(QloraLoraLinear), ctypes.POINTER(QloraLoraLinear),
                                     ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                     ctypes.POINTER(QloraMlpSaved), ctypes.c_void_p, ctypes.c_size_t,
                                     ctypes.c_void_p]),
    "qlora_mlp_bwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(QloraLoraLinear),
                                     ctypes.POINTER(QloraLoraLinear), ctypes.POINTER(QloraLoraLinear),
                                     ctypes.c_void_p, ctypes.POINTER(QloraMlpSaved), ctypes.c_void_p,
                                     ctypes.c_int64] + [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_mlp_bwd_ev": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(QloraLoraLinear),
                                        ctypes.POINTER(QloraLoraLinear), ctypes.POINTER(QloraLoraLinear),
                                        ctypes.c_void_p, ctypes.POINTER(QloraMlpSaved), ctypes.c_void_p,
                                        ctypes.c_int64] + [ctypes.c_void_p] * 8 +
                         [ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_mlp16_bwd_ev": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(QloraLoraLinear16),
                                          ctypes.POINTER(QloraLoraLinear16), ctypes.POINTER(QloraLoraLinear16),
                                          ctypes.c_void_p, ctypes.POINTER(QloraMlpSaved), ctypes.c_void_p,
                                          ctypes.c_int64] + [ctypes.c_void_p] * 8 +
                           [ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_last_device_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_test_inject_timeout": (ctypes.c_int, []),
    "qlora_test_set_grid_cap": (ctypes.c_int32, [ctypes.c_int32]),
    "qlora_test_shrink_next_slot_cap": (ctypes.c_int, []),
    "qlora_checked_build": (ctypes.c_int32, []),
    "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_set_tile_config": (ctypes.c_int32, [ctypes.c_int32]),
    "qlora_mlp_tile_config": (ctypes.c_int32, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]),
    "qlora_trace_begin": (ctypes.c_int, []),
    "qlora_trace_begin_only": (ctypes.c_int, [ctypes.c_char_p]),
    "qlora_trace_end": (ctypes.c_int32, [ctypes.POINTER(QloraTraceEntry), ctypes.c_int32]),
    "qlora_launch_count": (ctypes.c_uint64, []),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear), ctypes.c_void_p, ctypes.c_int64,
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_rmsnorm_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_float, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p]),
    "qlora_rmsnorm_bwd": (ctypes.c_int, [ctypes.c_void_p] * 4 + [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                                                 ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_qkv_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64] * 5 + [ctypes.c_int32]),
    "qlora_qkv_fwd": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear)] * 3 + [ctypes.c_void_p, ctypes.c_int64,
                                                                             ctypes.c_void_p, ctypes.c_void_p,
                                                                             ctypes.c_void_p, ctypes.c_size_t,
                                                                             ctypes.c_void_p]),
    "qlora_qkv_bwd": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear)] * 3 + [ctypes.c_void_p] * 3 +
                      [ctypes.c_int64] + [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear16_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                         ctypes.c_int32]),
    "qlora_mlp16_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                      ctypes.c_int32]),
    "qlora_linear16_fwd": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear16), ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p]),
    "qlora_linear16_bwd": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear16), ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_mlp16_fwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(QloraLoraLinear16),
                                       ctypes.POINTER(QloraLoraLinear16), ctypes.POINTER(QloraLoraLinear16),
                                       ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.POINTER(QloraMlpSaved), ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "qlora_mlp16_bwd": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(QloraLoraLinear16),
                                       ctypes.POINTER(QloraLoraLinear16), ctypes.POINTER(QloraLoraLinear16),
                                       ctypes.c_void_p, ctypes.POINTER(QloraMlpSaved), ctypes.c_void_p,
                                       ctypes.c_int64] + [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p]),
    "fp8_quantize_rows": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64] + [ctypes.c_void_p] * 3),
    "fp8_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64] + [ctypes.c_void_p] * 3),
    "fp8_matmul_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64] * 3),
    "fp8_matmul": (ctypes.c_int, [ctypes.POINTER(QloraFP8Rows), ctypes.POINTER(QloraFP8), ctypes.c_int64,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "fp8_matmul_t": (ctypes.c_int, [ctypes.POINTER(QloraFP8Rows), ctypes.POINTER(QloraFP8), ctypes.c_int64,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear8_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                        ctypes.c_int32]),
    "qlora_linear8_fwd": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear8), ctypes.c_void_p,
                                         ctypes.POINTER(QloraFP8Rows), ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_linear8_bwd": (ctypes.c_int, [ctypes.POINTER(QloraLoraLinear8), ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "qlora_add_rmsnorm_fwd": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_int64, ctypes.c_int64, ctypes.c_float,
                                                                     ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                                                     ctypes.POINTER(QloraFP8Rows), ctypes.c_void_p,
                                                                     ctypes.c_void_p]),
    "qlora_add_rmsnorm_bwd": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                                                     ctypes.c_void_p, ctypes.c_void_p]),
    "qlora_rope_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p]),
    "qlora_rope_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p]),
}


def _load(path):
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m qlora_fine_tuning_nf4_b200.build`")
    L = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


def lib():
    """Load libqlora.so, or libqlora_check.so under QLORA_LIBRARY=checked (raises if it has not been built)."""
    global _lib
    if _lib is None:
        choice = os.environ.get("QLORA_LIBRARY", "")
        if choice not in ("", "checked"):
            raise RuntimeError(f"QLORA_LIBRARY={choice!r}: expected unset or 'checked'")
        _lib = _load(CHECK_LIB_PATH if choice == "checked" else LIB_PATH)
    return _lib


_check_lib = None


def checked_lib():
    """Load the bounds-checked debug build, libqlora_check.so (same ABI; its
    kernels report out-of-range indices as QLORA_ERR_DEVICE instead of
    touching memory out of range)."""
    global _check_lib
    if _check_lib is None:
        _check_lib = _load(CHECK_LIB_PATH)
    return _check_lib


_normal_lib = None


def normal_lib():
    """Load the normal build, libqlora.so, whatever QLORA_LIBRARY selects."""
    global _normal_lib
    if _normal_lib is None:
        _normal_lib = _load(LIB_PATH)
    return _normal_lib


class use_library:
    """Context manager that routes every wrapper of this module to another
    build of the library (e.g. checked_lib()) and restores the previous one."""

    def __init__(self, L):
        self.L = L

    def __enter__(self):
        global _lib
        self.prev = lib()
        _lib = self.L
        return self.L

    def __exit__(self, *exc):
        global _lib
        _lib = self.prev
        return False


def _check(fn, status):
    if status != QLORA_OK:
        raise QloraError(fn, status)


# torch's own accessors of the current device and stream, without the Python layers above them (a call's host time
# is a good part of a small operator's: 28 -> 12 us for a norm of one token with four outputs)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing


def _stream():
    if _raw_stream is not None:
        return _raw_stream(_current_device())
    return torch.cuda.current_stream().cuda_stream


def _p(t):
    return 0 if t is None else t.data_ptr()


def _dev(t, name):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t


def _t(t, name, shape, dtype=torch.bfloat16):
    """Marshalling check of one tensor argument: contiguous, on the current
    CUDA device, of the expected dtype and shape.  The C ABI only sees raw
    pointers, so a host tensor or a short buffer must be caught here."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda
            and t.get_device() == _current_device()):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _rows(X, name="X"):
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor [M, features]")
    return X.shape


# ------------------------------------------------------------------ NF4 ----

@dataclass
class NF4Weight:
    codes: torch.Tensor   # uint8 [n_out * k_in / 2]
    absmax: torch.Tensor  # float32 [n_out * k_in / 64]
    n_out: int
    k_in: int

    def c(self):
        _t(self.codes, "codes", (self.n_out * self.k_in // 2,), torch.uint8)
        _t(self.absmax, "absmax", (self.n_out * self.k_in // 64,), torch.float32)
        return QloraNF4(self.codes.data_ptr(), self.absmax.data_ptr(), self.n_out, self.k_in)


def qlora_nf4_codebook():
    out = (ctypes.c_float * 16)()
    _check("qlora_nf4_codebook", lib().qlora_nf4_codebook(out))
    return [float(v) for v in out]


def nf4_quantize(w):
    """bf16 weight [n_out, k_in] on the GPU -> NF4Weight."""
    n_out, k_in = _rows(w, "w")
    _t(w, "w", (n_out, k_in))
    codes = torch.empty(n_out * k_in // 2, dtype=torch.uint8, device=w.device)
    absmax = torch.empty(n_out * k_in // 64, dtype=torch.float32, device=w.device)
    _check("nf4_quantize", lib().nf4_quantize(_p(w), n_out, k_in, _p(codes), _p(absmax), _stream()))
    return NF4Weight(codes, absmax, n_out, k_in)


def nf4_dequantize(w: NF4Weight, out=None):
    """NF4Weight -> bf16 [n_out, k_in] (bit-exact)."""
    if out is None:
        out = torch.empty(w.n_out, w.k_in, dtype=torch.bfloat16, device=w.codes.device)
    w.c()  # checks codes and absmax
    _t(out, "out", (w.n_out, w.k_in))
    _check("nf4_dequantize", lib().nf4_dequantize(_p(w.codes), _p(w.absmax), w.n_out, w.k_in, _p(out), _stream()))
    return out


# ---------------------------------------------------------- projections ----

@dataclass
class LoraLinear:
    w: NF4Weight
    A: torch.Tensor  # bf16 [k_in, r]
    B: torch.Tensor  # bf16 [r, n_out]
    scale: float

    def c(self):
        r = self.A.shape[1] if self.A.dim() == 2 else -1
        _t(self.A, "A", (self.w.k_in, r))
        _t(self.B, "B", (r, self.w.n_out))
        return QloraLoraLinear(self.w.c(), self.A.data_ptr(), self.B.data_ptr(), r, self.scale)


@dataclass
class LoraLinear16:
    """A projection with a frozen bf16 base weight (LoRA rather than QLoRA)."""
    w: torch.Tensor  # bf16 [n_out, k_in]
    A: torch.Tensor  # bf16 [k_in, r]
    B: torch.Tensor  # bf16 [r, n_out]
    scale: float

    @property
    def n_out(self):
        return self.w.shape[0]

    @property
    def k_in(self):
        return self.w.shape[1]

    def c(self):
        if self.w.dim() != 2:
            raise ValueError("w must be a 2-D bf16 tensor [n_out, k_in]")
        _t(self.w, "w", tuple(self.w.shape))
        r = self.A.shape[1] if self.A.dim() == 2 else -1
        _t(self.A, "A", (self.k_in, r))
        _t(self.B, "B", (r, self.n_out))
        return QloraLoraLinear16(self.w.data_ptr(), self.n_out, self.k_in, self.A.data_ptr(), self.B.data_ptr(),
                                 r, self.scale)


def _dims(lin):
    """(n_out, k_in) of an NF4 or a bf16 projection."""
    return (lin.w.n_out, lin.w.k_in) if isinstance(lin, LoraLinear) else (lin.n_out, lin.k_in)


_growth_streams = {}  # device index -> stream on which buffers are zeroed while the current stream is being captured


def _zeroed_outside_capture(nbytes):
    """Zeroed bytes while the current stream is being captured.  Made there they would belong to the graph: zeroed by
    each of its replays (with the status word in them) and by nothing before the first one, in memory that other
    graphs of the pool write to.  So they are made on a stream that is not captured, and zero on return.  A thread
    that captures may allocate and wait meanwhile in the relaxed capture mode only (CUDA's documentation of
    cuThreadExchangeStreamCaptureMode)."""
    exchange = ctypes.CDLL("libcuda.so.1").cuThreadExchangeStreamCaptureMode
    mode = ctypes.c_int(2)  # CU_STREAM_CAPTURE_MODE_RELAXED; the call leaves the mode that was set
    if exchange(ctypes.byref(mode)) != 0:
        raise RuntimeError("cuThreadExchangeStreamCaptureMode failed")
    try:
        dev = _current_device()
        if dev not in _growth_streams:
            _growth_streams[dev] = torch.cuda.Stream()
        with torch.cuda.stream(_growth_streams[dev]):
            buf = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        _growth_streams[dev].synchronize()
    finally:
        exchange(ctypes.byref(mode))
    return buf


class Workspace:
    """Caller-owned device workspace (zeroed once; grows on demand, also while its calls are being captured).

    One workspace serves calls whose GPU work does not overlap: calls on one stream, or graphs replayed one after
    the other, in any order.  Streams that run at the same time need one each.  It has to outlive the graphs that
    were captured with it; a buffer that calls were captured with stays alive after the workspace has grown, since
    a graph's replay still uses it."""

    def __init__(self, device="cuda"):
        self.device = device
        self.captured, self.kept = False, []
        self._make(256)

    def _make(self, nbytes):
        with torch.cuda.device(self.device):  # its current stream counts, where the buffer is made on another device
            self.apart = bool(_capturing())   # made on a stream of its own
            self.buf = (_zeroed_outside_capture(nbytes) if self.apart
                        else torch.zeros(nbytes, dtype=torch.uint8, device="cuda"))

    def get(self, nbytes):
        if self.buf.get_device() != _current_device():
            raise ValueError(f"the workspace is on {self.buf.device}, not on the current device cuda:{_current_device()}")
        if self.buf.numel() < nbytes:
            old = self.buf
            self._make(nbytes)
            if self.captured or self.apart:  # a graph's replays use it, or its error (if any) cannot be copied now
                self.kept.append(old)
            else:
                self.buf[:4].copy_(old[:4])  # an error recorded so far
            self.captured = False
        if not self.captured and _capturing():
            self.captured = True
        elif self.apart and not _capturing():
            self.buf.record_stream(torch.cuda.current_stream())  # its memory is not reused before this call is done
        return self.buf


def qlora_linear_workspace_bytes(M, K, N, r=16):
    return int(lib().qlora_linear_workspace_bytes(M, K, N, r))


def qlora_mlp_workspace_bytes(M, d, h, r=16):
    return int(lib().qlora_mlp_workspace_bytes(M, d, h, r))


def qlora_linear16_workspace_bytes(M, K, N, r=16):
    return int(lib().qlora_linear16_workspace_bytes(M, K, N, r))


def qlora_mlp16_workspace_bytes(M, d, h, r=16):
    return int(lib().qlora_mlp16_workspace_bytes(M, d, h, r))


def _linear_fwd(fn, wsq, lin, X, ws, Y, XA):
    M = _rows(X)[0]
    n_out, k_in = _dims(lin)
    r = lin.A.shape[1]
    if Y is None:
        Y = torch.empty(M, n_out, dtype=torch.bfloat16, device=X.device)
    if XA is None:
        XA = torch.empty(M, r, dtype=torch.bfloat16, device=X.device)
    _t(X, "X", (M, k_in))
    _t(Y, "Y", (M, n_out))
    _t(XA, "XA", (M, r))
    c = lin.c()
    buf = ws.get(wsq(M, k_in, n_out, r))
    _check(fn, getattr(lib(), fn)(ctypes.byref(c), _p(X), M, _p(Y), _p(XA), _p(buf), buf.numel(), _stream()))
    return Y, XA


def qlora_linear_fwd(lin: LoraLinear, X, ws: Workspace, Y=None, XA=None):
    return _linear_fwd("qlora_linear_fwd", qlora_linear_workspace_bytes, lin, X, ws, Y, XA)


def qlora_linear16_fwd(lin: LoraLinear16, X, ws: Workspace, Y=None, XA=None):
    return _linear_fwd("qlora_linear16_fwd", qlora_linear16_workspace_bytes, lin, X, ws, Y, XA)


def qlora_linear_fwd_noalloc(lin: LoraLinear, X, Y=None, XA=None):
    """qlora_linear_fwd without a workspace, for callers that cannot allocate
    device memory; its scratch is a fixed array inside the library (shared by
    all calls, so calls must not overlap on the GPU)."""
    M = _rows(X)[0]
    r = lin.A.shape[1]
    if Y is None:
        Y = torch.empty(M, lin.w.n_out, dtype=torch.bfloat16, device=X.device)
    if XA is None:
        XA = torch.empty(M, r, dtype=torch.bfloat16, device=X.device)
    _t(X, "X", (M, lin.w.k_in))
    _t(Y, "Y", (M, lin.w.n_out))
    _t(XA, "XA", (M, r))
    c = lin.c()
    _check("qlora_linear_fwd_noalloc", lib().qlora_linear_fwd_noalloc(ctypes.byref(c), _p(X), M, _p(Y), _p(XA),
                                                                      _stream()))
    return Y, XA


def _linear_bwd(fn, wsq, lin, X, XA, dY, ws, dX, dA, dB):
    M = _rows(X)[0]
    n_out, k_in = _dims(lin)
    r = lin.A.shape[1]
    if dX is None:
        dX = torch.empty(M, k_in, dtype=torch.bfloat16, device=X.device)
    if dA is None:
        dA = torch.empty_like(lin.A)
    if dB is None:
        dB = torch.empty_like(lin.B)
    _t(X, "X", (M, k_in))
    _t(XA, "XA", (M, r))
    _t(dY, "dY", (M, n_out))
    _t(dX, "dX", (M, k_in))
    _t(dA, "dA", (k_in, r))
    _t(dB, "dB", (r, n_out))
    c = lin.c()
    buf = ws.get(wsq(M, k_in, n_out, r))
    _check(fn, getattr(lib(), fn)(ctypes.byref(c), _p(X), _p(XA), _p(dY), M, _p(dX), _p(dA), _p(dB), _p(buf),
                                  buf.numel(), _stream()))
    return dX, dA, dB


def qlora_linear_bwd(lin: LoraLinear, X, XA, dY, ws: Workspace, dX=None, dA=None, dB=None):
    return _linear_bwd("qlora_linear_bwd", qlora_linear_workspace_bytes, lin, X, XA, dY, ws, dX, dA, dB)


def qlora_linear16_bwd(lin: LoraLinear16, X, XA, dY, ws: Workspace, dX=None, dA=None, dB=None):
    return _linear_bwd("qlora_linear16_bwd", qlora_linear16_workspace_bytes, lin, X, XA, dY, ws, dX, dA, dB)


def make_mlp_saved(M, h, r, device):
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=device)
    return {"E": e(M, h), "G": e(M, h), "H": e(M, h), "XA_g": e(M, r), "XA_u": e(M, r), "HA_d": e(M, r)}


def _saved_c(sv, M, h, r):
    for k in ("E", "G", "H"):
        _t(sv[k], k, (M, h))
    for k in ("XA_g", "XA_u", "HA_d"):
        _t(sv[k], k, (M, r))
    return QloraMlpSaved(*[sv[k].data_ptr() for k in ("E", "G", "H", "XA_g", "XA_u", "HA_d")])


def _mlp_dims(gate, up, down, d):
    h = _dims(gate)[0]
    if _dims(gate) != (h, d) or _dims(up) != (h, d) or _dims(down) != (d, h):
        raise ValueError(f"MLP weights must be gate, up [h, {d}] and down [{d}, h]")
    return h


def _mlp_fwd(fn, wsq, act, gate, up, down, X, ws, Y, saved):
    M, d = _rows(X)
    h = _mlp_dims(gate, up, down, d)
    r = gate.A.shape[1]
    if Y is None:
        Y = torch.empty(M, d, dtype=torch.bfloat16, device=X.device)
    if saved is None:
        saved = make_mlp_saved(M, h, r, X.device)
    _t(X, "X", (M, d))
    _t(Y, "Y", (M, d))
    g, u, dn, sv = gate.c(), up.c(), down.c(), _saved_c(saved, M, h, r)
    buf = ws.get(wsq(M, d, h, r))
    _check(fn, getattr(lib(), fn)(QLORA_ACT[act], ctypes.byref(g), ctypes.byref(u), ctypes.byref(dn), _p(X), M,
                                  _p(Y), ctypes.byref(sv), _p(buf), buf.numel(), _stream()))
    return Y, saved


def qlora_mlp_fwd(act, gate: LoraLinear, up: LoraLinear, down: LoraLinear, X, ws: Workspace, Y=None, saved=None):
    return _mlp_fwd("qlora_mlp_fwd", qlora_mlp_workspace_bytes, act, gate, up, down, X, ws, Y, saved)


def qlora_mlp16_fwd(act, gate: LoraLinear16, up: LoraLinear16, down: LoraLinear16, X, ws: Workspace, Y=None,
                    saved=None):
    return _mlp_fwd("qlora_mlp16_fwd", qlora_mlp16_workspace_bytes, act, gate, up, down, X, ws, Y, saved)


def _mlp_bwd(fn, wsq, act, gate, up, down, X, saved, dY, ws, grads, early_event=0):
    M, d = _rows(X)
    h = _mlp_dims(gate, up, down, d)
    r = gate.A.shape[1]
    if grads is None:
        grads = {"dX": torch.empty(M, d, dtype=torch.bfloat16, device=X.device),
                 "dA_g": torch.empty_like(gate.A), "dB_g": torch.empty_like(gate.B),
                 "dA_u": torch.empty_like(up.A), "dB_u": torch.empty_like(up.B),
                 "dA_d": torch.empty_like(down.A), "dB_d": torch.empty_like(down.B)}
    _t(X, "X", (M, d))
    _t(dY, "dY", (M, d))
    _t(grads["dX"], "dX", (M, d))
    for k, shp in (("dA_g", (d, r)), ("dB_g", (r, h)), ("dA_u", (d, r)), ("dB_u", (r, h)), ("dA_d", (h, r)),
                   ("dB_d", (r, d))):
        _t(grads[k], k, shp)
    g, u, dn, sv = gate.c(), up.c(), down.c(), _saved_c(saved, M, h, r)
    buf = ws.get(wsq(M, d, h, r))
    outs = [_p(grads[k]) for k in ("dX", "dA_g", "dB_g", "dA_u", "dB_u", "dA_d", "dB_d")]
    args = [QLORA_ACT[act], ctypes.byref(g), ctypes.byref(u), ctypes.byref(dn), _p(X), ctypes.byref(sv), _p(dY), M,
            *outs, _p(buf), buf.numel(), _stream()]
    if early_event:
        _check(fn + "_ev", getattr(lib(), fn + "_ev")(*args, ctypes.c_void_p(early_event)))
    else:
        _check(fn, getattr(lib(), fn)(*args))
    return grads


def qlora_mlp_bwd(act, gate: LoraLinear, up: LoraLinear, down: LoraLinear, X, saved, dY, ws: Workspace, grads=None,
                  early_event=0):
    """MLP backward; with `early_event` (a raw cudaEvent_t, e.g. torch.cuda.Event().cuda_event after its first
    record) the library records it once dA_d, dB_d, dB_g and dB_u are final (qlora_mlp_bwd_ev)."""
    return _mlp_bwd("qlora_mlp_bwd", qlora_mlp_workspace_bytes, act, gate, up, down, X, saved, dY, ws, grads,
                    early_event)


def qlora_mlp16_bwd(act, gate: LoraLinear16, up: LoraLinear16, down: LoraLinear16, X, saved, dY, ws: Workspace,
                    grads=None, early_event=0):
    return _mlp_bwd("qlora_mlp16_bwd", qlora_mlp16_workspace_bytes, act, gate, up, down, X, saved, dY, ws, grads,
                    early_event)


def qlora_rmsnorm_fwd(X, w, eps, plus_one=False, Y=None, rstd=None):
    """RMS layer norm of X [M, d] with gain w (or 1 + w): returns (Y, rstd)."""
    M, d = _rows(X)
    if Y is None:
        Y = torch.empty_like(X)
    if rstd is None:
        rstd = torch.empty(M, dtype=torch.float32, device=X.device)
    _t(X, "X", (M, d))
    _t(w, "w", (d,))
    _t(Y, "Y", (M, d))
    _t(rstd, "rstd", (M,), torch.float32)
    _check("qlora_rmsnorm_fwd", lib().qlora_rmsnorm_fwd(_p(X), _p(w), M, d, float(eps), int(bool(plus_one)), _p(Y),
                                                        _p(rstd), _stream()))
    return Y, rstd


def qlora_rmsnorm_bwd(X, w, rstd, dY, plus_one=False, dX=None):
    M, d = _rows(X)
    if dX is None:
        dX = torch.empty_like(X)
    _t(X, "X", (M, d))
    _t(w, "w", (d,))
    _t(rstd, "rstd", (M,), torch.float32)
    _t(dY, "dY", (M, d))
    _t(dX, "dX", (M, d))
    _check("qlora_rmsnorm_bwd", lib().qlora_rmsnorm_bwd(_p(X), _p(w), _p(rstd), _p(dY), M, d, int(bool(plus_one)),
                                                        _p(dX), _stream()))
    return dX


def qlora_qkv_workspace_bytes(M, K, nq, nk, nv, r=16):
    return int(lib().qlora_qkv_workspace_bytes(M, K, nq, nk, nv, r))


def qlora_qkv_fwd(q: LoraLinear, k: LoraLinear, v: LoraLinear, X, ws: Workspace, Y=None, XA=None):
    """Fused Q/K/V projection: Y = [Y_q | Y_k | Y_v] [M, nq + nk + nv], XA = [XA_q | XA_k | XA_v] [M, 3r]."""
    M, K = _rows(X)
    r = q.A.shape[1]
    nt = q.w.n_out + k.w.n_out + v.w.n_out
    if Y is None:
        Y = torch.empty(M, nt, dtype=torch.bfloat16, device=X.device)
    if XA is None:
        XA = torch.empty(M, 3 * r, dtype=torch.bfloat16, device=X.device)
    _t(X, "X", (M, K))
    _t(Y, "Y", (M, nt))
    _t(XA, "XA", (M, 3 * r))
    cq, ck, cv = q.c(), k.c(), v.c()
    buf = ws.get(qlora_qkv_workspace_bytes(M, K, q.w.n_out, k.w.n_out, v.w.n_out, r))
    _check("qlora_qkv_fwd", lib().qlora_qkv_fwd(ctypes.byref(cq), ctypes.byref(ck), ctypes.byref(cv), _p(X), M,
                                                _p(Y), _p(XA), _p(buf), buf.numel(), _stream()))
    return Y, XA


def qlora_qkv_bwd(q: LoraLinear, k: LoraLinear, v: LoraLinear, X, XA, dY, ws: Workspace, grads=None):
    M, K = _rows(X)
    r = q.A.shape[1]
    nt = q.w.n_out + k.w.n_out + v.w.n_out
    if grads is None:
        grads = {"dX": torch.empty(M, K, dtype=torch.bfloat16, device=X.device)}
        for n, l in (("q", q), ("k", k), ("v", v)):
            grads["dA_" + n] = torch.empty_like(l.A)
            grads["dB_" + n] = torch.empty_like(l.B)
    _t(X, "X", (M, K))
    _t(XA, "XA", (M, 3 * r))
    _t(dY, "dY", (M, nt))
    _t(grads["dX"], "dX", (M, K))
    for n, l in (("q", q), ("k", k), ("v", v)):
        _t(grads["dA_" + n], "dA_" + n, (K, r))
        _t(grads["dB_" + n], "dB_" + n, (r, l.w.n_out))
    cq, ck, cv = q.c(), k.c(), v.c()
    buf = ws.get(qlora_qkv_workspace_bytes(M, K, q.w.n_out, k.w.n_out, v.w.n_out, r))
    outs = [_p(grads[n]) for n in ("dX", "dA_q", "dB_q", "dA_k", "dB_k", "dA_v", "dB_v")]
    _check("qlora_qkv_bwd", lib().qlora_qkv_bwd(ctypes.byref(cq), ctypes.byref(ck), ctypes.byref(cv), _p(X), _p(XA),
                                                _p(dY), M, *outs, _p(buf), buf.numel(), _stream()))
    return grads


# ---------------------------------------------------------------- 8-bit ----

FP8_BLOCK = 128  # columns of a row, or rows and columns of a weight, that share a scale


def _blocks(n):
    return -(-n // FP8_BLOCK)


@dataclass
class FP8Rows:
    """Rows [M, K] in 8 bits: value = codes[m, k] * scale[k // 128, m]."""
    codes: torch.Tensor  # float8_e4m3fn [M, K]
    scale: torch.Tensor  # float32 [ceil(K / 128), M]

    def c(self, name="rows", shape=None):
        if not isinstance(self.codes, torch.Tensor) or self.codes.dim() != 2:
            raise ValueError(f"{name}.codes must be a 2-D float8_e4m3fn tensor [M, K]")
        M, K = shape or self.codes.shape
        _t(self.codes, name + ".codes", (M, K), torch.float8_e4m3fn)
        _t(self.scale, name + ".scale", (_blocks(K), M), torch.float32)
        return QloraFP8Rows(self.codes.data_ptr(), self.scale.data_ptr())


@dataclass
class FP8Weight:
    """Frozen weight [n_out, k_in] in 8 bits: value = codes[n, k] * scale[n // 128, k // 128]."""
    codes: torch.Tensor  # float8_e4m3fn [n_out, k_in]
    scale: torch.Tensor  # float32 [ceil(n_out / 128), ceil(k_in / 128)]

    @property
    def n_out(self):
        return self.codes.shape[0]

    @property
    def k_in(self):
        return self.codes.shape[1]

    def c(self):
        codes, scale = self.codes, self.scale
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise ValueError("codes must be a 2-D float8_e4m3fn tensor [n_out, k_in]")
        n, k = codes.shape
        _t(codes, "codes", (n, k), torch.float8_e4m3fn)
        _t(scale, "scale", (_blocks(n), _blocks(k)), torch.float32)
        return QloraFP8(codes.data_ptr(), scale.data_ptr(), n, k)


def _empty_rows(M, K, like):
    return FP8Rows(like.new_empty((M, K), dtype=torch.float8_e4m3fn),
                   like.new_empty((_blocks(K), M), dtype=torch.float32))


def fp8_quantize_rows(X, out: FP8Rows = None):
    """bf16 rows [M, K] -> FP8Rows (one power-of-two scale per 128 columns)."""
    M, K = _rows(X)
    _t(X, "X", (M, K))
    if out is None:
        out = _empty_rows(M, K, X)
    c = out.c("out", (M, K))
    _check("fp8_quantize_rows", lib().fp8_quantize_rows(_p(X), M, K, c.codes, c.scale, _stream()))
    return out


def fp8_quantize(w):
    """bf16 weight [n_out, k_in] on the GPU -> FP8Weight (one power-of-two scale per 128 x 128 block)."""
    n_out, k_in = _rows(w, "w")
    _t(w, "w", (n_out, k_in))
    q = FP8Weight(torch.empty(n_out, k_in, dtype=torch.float8_e4m3fn, device=w.device),
                  torch.empty(_blocks(n_out), _blocks(k_in), dtype=torch.float32, device=w.device))
    _check("fp8_quantize", lib().fp8_quantize(_p(w), n_out, k_in, _p(q.codes), _p(q.scale), _stream()))
    return q


def _call_ws(fn, ws, need, args):
    """One call that ends in (workspace, its bytes, stream).  The library checks the size before it enqueues anything,
    so the size is asked for only when the workspace at hand is too small."""
    f = getattr(lib(), fn)
    buf = ws.get(0)
    status = f(*args, buf.data_ptr(), buf.numel(), _stream())
    if status == 4:  # QLORA_ERR_WORKSPACE_TOO_SMALL
        buf = ws.get(need())
        status = f(*args, buf.data_ptr(), buf.numel(), _stream())
    _check(fn, status)


def fp8_matmul_workspace_bytes(M, K, N):
    """For M rows; fewer rows may need more (a split reduction's partial sums), so ask for every M that is used."""
    return int(lib().fp8_matmul_workspace_bytes(M, K, N))


def _fp8_matmul(fn, x, w, ws, out, transposed):
    if not isinstance(x, FP8Rows) or not isinstance(w, FP8Weight):
        raise TypeError(f"{fn} takes FP8Rows and FP8Weight")
    if not isinstance(x.codes, torch.Tensor) or x.codes.dim() != 2:
        raise ValueError("x.codes must be a 2-D float8_e4m3fn tensor")
    cw = w.c()
    n_out, k_in = w.codes.shape
    red, cols = (n_out, k_in) if transposed else (k_in, n_out)
    M = x.codes.shape[0]
    cx = x.c("x", (M, red))
    if out is None:
        out = x.codes.new_empty((M, cols), dtype=torch.bfloat16)
    else:
        _t(out, "out", (M, cols))
    _call_ws(fn, ws, lambda: fp8_matmul_workspace_bytes(M, k_in, n_out),
             (ctypes.byref(cx), ctypes.byref(cw), M, out.data_ptr()))
    return out


def fp8_matmul(x: FP8Rows, w: FP8Weight, ws: Workspace, Y=None):
    """Y = x W^T [M, n_out] in bf16 from x [M, k_in]."""
    return _fp8_matmul("fp8_matmul", x, w, ws, Y, False)


def fp8_matmul_t(dY: FP8Rows, w: FP8Weight, ws: Workspace, dX=None):
    """dX = dY W [M, k_in] in bf16 from dY [M, n_out]."""
    return _fp8_matmul("fp8_matmul_t", dY, w, ws, dX, True)


@dataclass
class LoraLinear8:
    """A projection with a frozen e4m3 base weight."""
    w: FP8Weight
    A: torch.Tensor  # bf16 [k_in, r]
    B: torch.Tensor  # bf16 [r, n_out]
    scale: float

    def c(self):
        A, B = self.A, self.B
        cw = self.w.c()
        n_out, k_in = self.w.codes.shape
        r = A.shape[1] if A.dim() == 2 else -1
        _t(A, "A", (k_in, r))
        _t(B, "B", (r, n_out))
        return QloraLoraLinear8(cw, A.data_ptr(), B.data_ptr(), r, self.scale)


def qlora_linear8_workspace_bytes(M, K, N, r=16):
    """For M rows; fewer rows may need more, so ask for every M that is used."""
    return int(lib().qlora_linear8_workspace_bytes(M, K, N, r))


def qlora_linear8_fwd(lin: LoraLinear8, X, ws: Workspace, Y=None, XA=None, X8: FP8Rows = None):
    """Y = q(X) W^T + s (X A) B, XA = X A; X8 = X already in 8 bits (else the call quantises it)."""
    M = _rows(X)[0]
    c = lin.c()
    (k_in, r), n_out = lin.A.shape, lin.B.shape[1]
    _t(X, "X", (M, k_in))
    Y = X.new_empty((M, n_out)) if Y is None else _t(Y, "Y", (M, n_out))
    XA = X.new_empty((M, r)) if XA is None else _t(XA, "XA", (M, r))
    c8 = X8.c("X8", (M, k_in)) if X8 is not None else None
    _call_ws("qlora_linear8_fwd", ws, lambda: qlora_linear8_workspace_bytes(M, k_in, n_out, r),
             (ctypes.byref(c), X.data_ptr(), ctypes.byref(c8) if c8 else None, M, Y.data_ptr(), XA.data_ptr()))
    return Y, XA


def qlora_linear8_bwd(lin: LoraLinear8, X, XA, dY, ws: Workspace, dX=None, dA=None, dB=None):
    M = _rows(X)[0]
    c = lin.c()
    (k_in, r), n_out = lin.A.shape, lin.B.shape[1]
    _t(X, "X", (M, k_in))
    _t(XA, "XA", (M, r))
    _t(dY, "dY", (M, n_out))
    dX = X.new_empty((M, k_in)) if dX is None else _t(dX, "dX", (M, k_in))
    dA = X.new_empty((k_in, r)) if dA is None else _t(dA, "dA", (k_in, r))
    dB = X.new_empty((r, n_out)) if dB is None else _t(dB, "dB", (r, n_out))
    _call_ws("qlora_linear8_bwd", ws, lambda: qlora_linear8_workspace_bytes(M, k_in, n_out, r),
             (ctypes.byref(c), X.data_ptr(), XA.data_ptr(), dY.data_ptr(), M, dX.data_ptr(), dA.data_ptr(),
              dB.data_ptr()))
    return dX, dA, dB


# -------------------------------------------------- residual add + norm ----

def qlora_add_rmsnorm_fwd(X, R, w, eps, plus_one=False, H=None, Y=None, rstd=None, quantize=False, Y8: FP8Rows = None,
                          want_y=True):
    """H = X + R (R None: H is X), RMS norm of H with gain w (or 1 + w): returns (H, Y, rstd, Y8).

    Y8 (FP8Rows of Y) is written with quantize=True or where it is given, else None; Y is None with
    want_y=False.  H may be X or R."""
    M, d = _rows(X)
    if R is None and H is not None and H is not X:
        raise ValueError("H is X itself where R is None")
    _t(X, "X", (M, d))
    if R is not None:
        _t(R, "R", (M, d))
        H = torch.empty_like(X) if H is None else _t(H, "H", (M, d))
    _t(w, "w", (d,))
    if Y is not None:
        _t(Y, "Y", (M, d))
    elif want_y:
        Y = torch.empty_like(X)
    rstd = X.new_empty((M,), dtype=torch.float32) if rstd is None else _t(rstd, "rstd", (M,), torch.float32)
    c8 = None
    if Y8 is not None:
        c8 = Y8.c("Y8", (M, d))
    elif quantize:
        Y8 = _empty_rows(M, d, X)
        c8 = QloraFP8Rows(Y8.codes.data_ptr(), Y8.scale.data_ptr())
    _check("qlora_add_rmsnorm_fwd", lib().qlora_add_rmsnorm_fwd(
        _p(X), _p(R), _p(w), M, d, float(eps), int(bool(plus_one)), _p(None if R is None else H), _p(Y),
        ctypes.byref(c8) if c8 else None, _p(rstd), _stream()))
    return X if R is None else H, Y, rstd, Y8


def qlora_add_rmsnorm_bwd(H, w, rstd, dY, dH=None, plus_one=False, dX=None):
    """Gradient of X and of R: dH (what reaches H past the norm) plus the norm's.  dX may be dY or dH."""
    M, d = _rows(H, "H")
    _t(H, "H", (M, d))
    _t(w, "w", (d,))
    _t(rstd, "rstd", (M,), torch.float32)
    _t(dY, "dY", (M, d))
    if dH is not None:
        _t(dH, "dH", (M, d))
    dX = torch.empty_like(H) if dX is None else _t(dX, "dX", (M, d))
    _check("qlora_add_rmsnorm_bwd", lib().qlora_add_rmsnorm_bwd(_p(H), _p(w), _p(rstd), _p(dY), _p(dH), M, d,
                                                                int(bool(plus_one)), _p(dX), _stream()))
    return dX


# ----------------------------------------------------------------- rope ----

@dataclass
class RopePlan:
    """Rotary frequencies of a model: pair i turns turns[i] / 2^64 of a circle per position."""
    turns: torch.Tensor  # int64 [rot / 2], the bits of the 64-bit fractions
    rot: int             # rotated elements of a head
    factor: float        # cosines and sines are multiplied by it


def rope_frequencies(rot, base=10000.0, scaling=None):
    """([radians per position of each pair], factor) in 64 bits.

    base^(-2i / rot), changed by `scaling`, a dict whose "type" is
      "linear"  frequencies / factor
      "ntk"     base * factor^(rot / (rot - 2)): the slowest pair is stretched by factor, the fastest kept
      "llama3"  pairs that turn less than low_freq_factor times in original_max_position are divided by
                factor, those above high_freq_factor times kept, a linear blend between
      "yarn"    pairs below beta_slow turns in original_max_position divided by factor, above beta_fast kept,
                a linear ramp over the pair index between; cosines and sines times attention_factor
                (0.1 ln(factor) + 1 unless given)."""
    if not isinstance(rot, int) or rot <= 0 or rot % 2:
        raise ValueError(f"rot must be a positive even integer, got {rot!r}")
    base = float(base)
    if not (base > 0.0 and math.isfinite(base)):
        raise ValueError(f"base must be positive, got {base!r}")
    s = dict(scaling or {"type": "none"})
    kind = s.pop("type", None)
    fields = {"none": (), "linear": ("factor",), "ntk": ("factor",),
              "llama3": ("factor", "low_freq_factor", "high_freq_factor", "original_max_position"),
              "yarn": ("factor", "original_max_position")}
    if kind not in fields:
        raise ValueError(f"unknown rope scaling {kind!r}: expected one of {sorted(fields)}")
    optional = {"beta_fast": 32.0, "beta_slow": 1.0, "attention_factor": None} if kind == "yarn" else {}
    missing, extra = set(fields[kind]) - set(s), set(s) - set(fields[kind]) - set(optional)
    if missing or extra:
        raise ValueError(f"rope scaling {kind!r}: missing {sorted(missing)}, not understood {sorted(extra)}")
    f = float(s.get("factor", 1.0))
    if not (f > 0.0 and math.isfinite(f)):
        raise ValueError(f"rope scaling factor must be positive, got {f!r}")
    if kind == "ntk":
        if rot == 2:
            raise ValueError("rope scaling 'ntk' needs more than one pair")
        base *= f ** (rot / (rot - 2))
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    factor = 1.0
    if kind == "linear":
        freq = [w / f for w in freq]
    elif kind == "llama3":
        lo, hi, n = float(s["low_freq_factor"]), float(s["high_freq_factor"]), float(s["original_max_position"])
        if not (hi > lo):
            raise ValueError("rope scaling 'llama3': high_freq_factor must be above low_freq_factor")
        blend = [min(1.0, max(0.0, (n * w / (2 * math.pi) - lo) / (hi - lo))) for w in freq]
        freq = [w * b + w / f * (1.0 - b) for w, b in zip(freq, blend)]
    elif kind == "yarn":
        n, opt = float(s["original_max_position"]), {**optional, **s}
        if not (n > 0.0 and base > 1.0):
            raise ValueError("rope scaling 'yarn' needs original_max_position > 0 and base > 1")
        # the (real) pair index that turns `t` times in n positions: n base^(-2i / rot) = 2 pi t
        index = lambda t: rot * math.log(n / (2 * math.pi * t)) / (2 * math.log(base))
        lo = max(math.floor(index(float(opt["beta_fast"]))), 0)
        hi = min(math.ceil(index(float(opt["beta_slow"]))), rot - 1)
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot // 2)]
        freq = [w / f * r + w * (1.0 - r) for w, r in zip(freq, ramp)]
        a = opt["attention_factor"]
        factor = (0.1 * math.log(f) + 1.0 if f > 1.0 else 1.0) if a is None else float(a)
    return freq, factor


def rope_plan(rot, base=10000.0, scaling=None, device="cuda"):
    """RopePlan of `rope_frequencies(rot, base, scaling)` on the GPU; made once per model.

    The frequencies are binary64 numbers, so an entry is off by (ln(base) + 4) 2^-53 of itself and half a unit of 2^-64
    turns: at position 2^20 that is below 2^-34 turns, at 2^31 about 2^-24 for the fastest pairs."""
    freq, factor = rope_frequencies(rot, base, scaling)
    bits = []
    for w in freq:
        t = int(round(w / (2 * math.pi) * 2.0 ** 64)) & (2 ** 64 - 1)
        bits.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    return RopePlan(torch.tensor(bits, dtype=torch.int64, device=device), rot, factor)


def _rope_rows(t, name, cols):
    """Check of a bf16 [M, cols] operand whose rows may be a slice of wider ones; returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2 or t.shape[1] != cols:
        raise ValueError(f"{name} must have shape [M, {cols}], got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{torch.cuda.current_device()}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) < cols):
        raise ValueError(f"{name} must have contiguous rows that do not overlap, got strides {t.stride()}")
    return t.stride(0) if t.shape[0] > 1 else cols


def _rope(fn, X, heads, head_dim, plan, positions, seq_len, interleaved, out):
    heads, head_dim = int(heads), int(head_dim)
    cols = heads * head_dim
    ldx = _rope_rows(X, "X", cols)
    M = X.shape[0]
    if out is None:
        out, ldo = X.new_empty((M, cols)), cols
    else:
        ldo = _rope_rows(out, "out", cols)
        if out.shape[0] != M:
            raise ValueError(f"out must have {M} rows, got {out.shape[0]}")
    if M > 0 and not (out.data_ptr() == X.data_ptr() and ldo == ldx):
        # in place, apart in memory, or other columns of the same rows
        a, b = X.data_ptr() // 2, out.data_ptr() // 2
        if a < b + (M - 1) * ldo + cols and b < a + (M - 1) * ldx + cols:
            if ldx != ldo or not cols <= (b - a) % ldx <= ldx - cols:
                raise ValueError("out overlaps X without being X")
    _t(plan.turns, "plan.turns", (plan.rot // 2,), torch.int64)
    if positions is not None:
        if seq_len:
            raise ValueError("give positions or seq_len, not both")
        _t(positions, "positions", (M,), torch.int64)
    _check(fn, getattr(lib(), fn)(_p(X), M, ldx, heads, head_dim, _p(plan.turns), plan.rot, int(bool(interleaved)),
                                  plan.factor, _p(positions), int(seq_len), _p(out), ldo, _stream()))
    return out


def qlora_rope_fwd(X, heads, head_dim, plan: RopePlan, positions=None, seq_len=0, interleaved=False, out=None):
    """Rotary positions on X [M, heads * head_dim], whose rows may be a slice of wider ones (the q and k
    columns of qlora_qkv_fwd's Y).  Row m has positions[m] (int64), else m % seq_len (m if 0).  out=X rotates
    in place."""
    return _rope("qlora_rope_fwd", X, heads, head_dim, plan, positions, seq_len, interleaved, out)


def qlora_rope_bwd(dY, heads, head_dim, plan: RopePlan, positions=None, seq_len=0, interleaved=False, out=None):
    """The gradient of qlora_rope_fwd's X: the transposed rotation of dY."""
    return _rope("qlora_rope_bwd", dY, heads, head_dim, plan, positions, seq_len, interleaved, out)


# ------------------------------------------------------------ utilities ----

def qlora_test_inject_timeout():
    """Arms the library's one-shot timeout injection (test hook; see include/qlora.h)."""
    _check("qlora_test_inject_timeout", lib().qlora_test_inject_timeout())


def qlora_test_shrink_next_slot_cap():
    """Arms the one-shot plan-mismatch hook (test only; see include/qlora.h)."""
    _check("qlora_test_shrink_next_slot_cap", lib().qlora_test_shrink_next_slot_cap())


def qlora_checked_build():
    return int(lib().qlora_checked_build())


def qlora_test_set_grid_cap(max_ctas):
    """Caps the CTAs of every persistent launch (test hook; 0 = no cap); returns the previous cap."""
    return int(lib().qlora_test_set_grid_cap(int(max_ctas)))


def qlora_last_device_status(ws: Workspace):
    """The error that calls with this workspace have recorded since it was last asked for (0: none), a timeout before
    any other; waits for the current stream."""
    found = [int(lib().qlora_last_device_status(_p(b), _stream())) for b in (ws.buf, *ws.kept)]
    return 6 if 6 in found else max(found)  # QLORA_ERR_TIMEOUT


def qlora_status_string(status):
    return lib().qlora_status_string(status).decode()


TILE_CONFIGS = {0: "automatic", 1: "1 CTA, 128x256", 2: "CTA pair, 256x256", 3: "CTA pair, 512x128",
                4: "CTA pair, 256x256, staged bf16 weight"}


def qlora_set_tile_config(tiles):
    return int(lib().qlora_set_tile_config(tiles))


def qlora_mlp_tile_config(M, d, h, r=16):
    """The tile configuration the NF4 MLP calls use for these sizes under the current setting."""
    return int(lib().qlora_mlp_tile_config(M, d, h, r))


def qlora_launch_count():
    return int(lib().qlora_launch_count())


def qlora_trace_begin(only=None):
    """Start tracing every kernel launch, or only the kernel named `only`."""
    if only is None:
        _check("qlora_trace_begin", lib().qlora_trace_begin())
    else:
        _check("qlora_trace_begin_only", lib().qlora_trace_begin_only(only.encode()))


def qlora_trace_end(max_entries=64):
    arr = (QloraTraceEntry * max_entries)()
    n = int(lib().qlora_trace_end(arr, max_entries))
    if n < 0:
        raise QloraError("qlora_trace_end", 5)
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms)) for i in range(min(n, max_entries))}
