"""B200 (sm_100a) FP8 W8A8 linear layer: Python binding of libfp8q.so.

The functions here carry the names of the C entry points declared in
include/fp8q.h and only marshal arguments: torch tensors supply device memory
and the current CUDA stream, every step of the computation runs in the
library's CUDA kernels.  There is no CPU fallback; without the built library
(or without a GPU) the calls raise.

    Wq, w_scale = fp8_quant_weight(W, mode)      # once per layer
    Xq, x_scale = fp8_quant_act(X, mode)         # every forward
    Y = fp8_linear(Xq, x_scale, Wq, w_scale, mode)

mode: CHANNEL_TOKEN (per-output-channel weights, per-token activations, the
FP8-Dynamic scheme) or BLOCK128 (128x128 weight blocks, 128-groups of
activations, the FP8-Block scheme).
"""
from __future__ import annotations

import ctypes
import importlib.util
import operator
import os
from typing import Optional, Tuple

import torch

from .policy import DEFAULT_IGNORE, should_quantize  # noqa: F401

CHANNEL_TOKEN = 0
BLOCK128 = 1
SCALE_BF16 = 0x10      # option OR'ed into a quantizer's mode: scales rounded to bf16 before the codes

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_MISALIGNED = 3
ERR_CUDA = 4
ERR_DEVICE_TIMEOUT = 5

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8q.so")
BINDING_PATH = os.path.join(_HERE, "_kv4_binding.so")

_lib = None


class FP8QError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """Load libfp8q.so (built in-tree by build.py); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libfp8q.so not built ({LIB_PATH}); run "
                              "python -m fp8_w8a8_quantized_amax_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        L.fp8_quant_weight.argtypes = [P, I, I, I, ctypes.c_int, P, I, P, P]
        L.fp8_quant_weight.restype = ctypes.c_int
        L.fp8_quant_act.argtypes = [P, I, I, I, ctypes.c_int, P, I, P, P]
        L.fp8_quant_act.restype = ctypes.c_int
        L.fp8_rmsnorm_quant_act.argtypes = [P, P, I, I, I, ctypes.c_float, P, I, P, P, P]
        L.fp8_rmsnorm_quant_act.restype = ctypes.c_int
        L.fp8_quant_act_static.argtypes = [P, I, I, I, ctypes.c_float, P, I, P, P]
        L.fp8_quant_act_static.restype = ctypes.c_int
        L.fp8_calibrate_static_scale.argtypes = [P, I, I, I, ctypes.c_double, ctypes.c_double, P, P, P]
        L.fp8_calibrate_static_scale.restype = ctypes.c_int
        L.fp8_linear_swiglu.argtypes = [P, P, P, P, P, P, I, I, I, P, I, P]
        L.fp8_linear_swiglu.restype = ctypes.c_int
        L.fp8_linear_w8a16.argtypes = [P, I, P, P, I, I, I, P, I, P, S, P]
        L.fp8_linear_w8a16.restype = ctypes.c_int
        L.fp8_linear_w8a16_workspace_size.argtypes = [I, I, I]
        L.fp8_linear_w8a16_workspace_size.restype = S
        L.fp8_linear.argtypes = [P, P, P, P, I, I, I, ctypes.c_int, P, I, P, S, P]
        L.fp8_linear.restype = ctypes.c_int
        L.fp8_linear_workspace_size.argtypes = [I, I, I, ctypes.c_int]
        L.fp8_linear_workspace_size.restype = S
        D, F, N = ctypes.c_double, ctypes.c_float, ctypes.c_int
        L.fp8q_rope_frequencies.argtypes = [P, I, D, P]
        L.fp8q_rope_frequencies.restype = N
        L.fp8q_rope.argtypes = [P, I, I, I, I, I, P, P, I, N, F, P, I, I, P]
        L.fp8q_rope.restype = N
        L.fp8q_kv4_page_bytes.argtypes = [I, I, I]
        L.fp8q_kv4_page_bytes.restype = S
        L.fp8q_kv4_append.argtypes = [P, P, I, I, P, I, I, P, I, P, P, I, N, F, P]
        L.fp8q_kv4_append.restype = N
        L.fp8q_kv4_read.argtypes = [P, P, I, P, I, I, P, I, I, P]
        L.fp8q_kv4_read.restype = N
        L.fp8q_kv4_attention_workspace_size.argtypes = [P, I, I, I, I]
        L.fp8q_kv4_attention_workspace_size.restype = S
        L.fp8q_kv4_attention.argtypes = [P, P, I, I, I, I, P, I, I, P, P, I, I, F, N, I, P, I, I, P, P, S, P]
        L.fp8q_kv4_attention.restype = N
        L.fp8q_status_string.argtypes = [ctypes.c_int]
        L.fp8q_status_string.restype = ctypes.c_char_p
        L.fp8q_device_error.argtypes = [ctypes.c_int]
        L.fp8q_device_error.restype = ctypes.c_int
        L.fp8q_version.argtypes = []
        L.fp8q_version.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fp8q_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise FP8QError(status, what)


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _require_cuda(t: torch.Tensor, name: str, dtype) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit stride in the last dimension")


def _numel(shape) -> int:
    n = 1
    for d in shape:
        n *= int(d)
    return n


def _require_like(t: Optional[torch.Tensor], name: str, dtype, min_numel: int, ref: torch.Tensor) -> None:
    """A scale vector or scratch buffer handed to a kernel: on ref's CUDA device,
    of `dtype`, contiguous, with at least min_numel elements.  (A host tensor
    would reach the kernel as a host pointer.)"""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or t.device != ref.device:
        raise ValueError(f"{name} must be a CUDA tensor on {ref.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {min_numel}")


def _require_out(t: torch.Tensor, name: str, dtype, shape, ref: torch.Tensor) -> None:
    """An output matrix: on ref's CUDA device, of `dtype` and `shape`, rows with unit stride."""
    if not t.is_cuda or t.device != ref.device:
        raise ValueError(f"{name} must be a CUDA tensor on {ref.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape) or (t.dim() == 2 and t.stride(1) != 1):
        raise ValueError(f"{name} must be {tuple(shape)} with unit stride in the last dimension")


def scale_shape_weight(N: int, K: int, mode: int) -> Tuple[int, ...]:
    return (N,) if (mode & ~SCALE_BF16) == CHANNEL_TOKEN else ((N + 127) // 128, K // 128)


def scale_shape_act(M: int, K: int, mode: int) -> Tuple[int, ...]:
    return (M,) if (mode & ~SCALE_BF16) == CHANNEL_TOKEN else (M, K // 128)


def fp8_quant_weight(W: torch.Tensor, mode: int = CHANNEL_TOKEN,
                     out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """W bf16 [N, K] -> (Wq uint8 [N, K] E4M3 codes, w_scale fp32 [N] or [N/128, K/128])."""
    _require_cuda(W, "W", torch.bfloat16)
    N, K = W.shape
    if out is None:
        Wq = torch.empty((N, K), dtype=torch.uint8, device=W.device)
        ws = torch.empty(scale_shape_weight(N, K, mode), dtype=torch.float32, device=W.device)
    else:
        Wq, ws = out
        _require_out(Wq, "Wq", torch.uint8, (N, K), W)
        _require_like(ws, "w_scale", torch.float32, _numel(scale_shape_weight(N, K, mode)), W)
    st = lib().fp8_quant_weight(_ptr(W), N, K, W.stride(0), int(mode), _ptr(Wq), Wq.stride(0),
                                _ptr(ws), _stream(W))
    _check(st, "fp8_quant_weight")
    return Wq, ws


def fp8_quant_act(X: torch.Tensor, mode: int = CHANNEL_TOKEN,
                  out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """X bf16 [M, K] -> (Xq uint8 [M, K], x_scale fp32 [M] or [M, K/128])."""
    _require_cuda(X, "X", torch.bfloat16)
    M, K = X.shape
    if out is None:
        Xq = torch.empty((M, K), dtype=torch.uint8, device=X.device)
        xs = torch.empty(scale_shape_act(M, K, mode), dtype=torch.float32, device=X.device)
    else:
        Xq, xs = out
        _require_out(Xq, "Xq", torch.uint8, (M, K), X)
        _require_like(xs, "x_scale", torch.float32, _numel(scale_shape_act(M, K, mode)), X)
    st = lib().fp8_quant_act(_ptr(X), M, K, X.stride(0), int(mode), _ptr(Xq), Xq.stride(0),
                             _ptr(xs), _stream(X))
    _check(st, "fp8_quant_act")
    return Xq, xs


def fp8_rmsnorm_quant_act(X: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5,
                          out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, return_rstd: bool = False):
    """RMSNorm(X) * gamma in bf16, quantized per token, in one pass.
    X bf16 [M, K], gamma bf16 [K] -> (Xq uint8 [M, K], x_scale fp32 [M][, rstd fp32 [M]])."""
    _require_cuda(X, "X", torch.bfloat16)
    M, K = X.shape
    if not gamma.is_cuda or gamma.device != X.device or gamma.dtype != torch.bfloat16 or gamma.numel() != K \
            or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous bf16 CUDA tensor of K elements on X's device")
    if out is None:
        Xq = torch.empty((M, K), dtype=torch.uint8, device=X.device)
        xs = torch.empty((M,), dtype=torch.float32, device=X.device)
    else:
        Xq, xs = out
        _require_out(Xq, "Xq", torch.uint8, (M, K), X)
        _require_like(xs, "x_scale", torch.float32, M, X)
    rstd = torch.empty((M,), dtype=torch.float32, device=X.device) if return_rstd else None
    st = lib().fp8_rmsnorm_quant_act(_ptr(X), _ptr(gamma), M, K, X.stride(0), float(eps), _ptr(Xq), Xq.stride(0),
                                     _ptr(xs), _ptr(rstd), _stream(X))
    _check(st, "fp8_rmsnorm_quant_act")
    return (Xq, xs, rstd) if return_rstd else (Xq, xs)


def fp8_quant_act_static(X: torch.Tensor, scale: float, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """X bf16 [M, K] coded with one fixed scale -> (Xq uint8 [M, K], x_scale fp32 [M] filled with scale)."""
    _require_cuda(X, "X", torch.bfloat16)
    M, K = X.shape
    if out is None:
        Xq = torch.empty((M, K), dtype=torch.uint8, device=X.device)
        xs = torch.empty((M,), dtype=torch.float32, device=X.device)
    else:
        Xq, xs = out
        _require_out(Xq, "Xq", torch.uint8, (M, K), X)
        if xs is not None:
            _require_like(xs, "x_scale", torch.float32, M, X)
    st = lib().fp8_quant_act_static(_ptr(X), M, K, X.stride(0), float(scale), _ptr(Xq), Xq.stride(0), _ptr(xs),
                                    _stream(X))
    _check(st, "fp8_quant_act_static")
    return Xq, xs


CALIB_HIST_BINS = 65536


def calibrate_static_scale(X: torch.Tensor, lo: float = 0.001, hi: float = 0.999,
                           hist: Optional[torch.Tensor] = None) -> float:
    """Offline calibration of a static scale (fp8_calibrate_static_scale): the
    larger magnitude of X's lo and hi quantiles, / 448, in fp32; 1.0 for a
    zero range.  X bf16 [M, K] on the GPU.  `hist`: a zero-filled int32
    device buffer of 65536 counts (allocated here when None; left zero)."""
    _require_cuda(X, "X", torch.bfloat16)
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M, K]")
    M, K = X.shape
    if hist is None:
        hist = torch.zeros(CALIB_HIST_BINS, dtype=torch.int32, device=X.device)
    _require_like(hist, "hist", torch.int32, CALIB_HIST_BINS, X)
    scale = torch.empty((), dtype=torch.float32, device=X.device)
    st = lib().fp8_calibrate_static_scale(_ptr(X), M, K, X.stride(0), float(lo), float(hi), _ptr(hist), _ptr(scale),
                                          _stream(X))
    _check(st, "fp8_calibrate_static_scale")
    return float(scale.item())


def fp8_linear_swiglu(Xq: torch.Tensor, x_scale: torch.Tensor, Wq_gate: torch.Tensor, w_scale_gate: torch.Tensor,
                      Wq_up: torch.Tensor, w_scale_up: torch.Tensor,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16(bf16(silu(g)) * u) of the gate and up projections (channel/token
    scales), g and u never written.  -> Y bf16 [M, N]."""
    _require_cuda(Xq, "Xq", torch.uint8)
    _require_cuda(Wq_gate, "Wq_gate", torch.uint8)
    _require_cuda(Wq_up, "Wq_up", torch.uint8)
    M, K = Xq.shape
    N = Wq_gate.shape[0]
    if Wq_gate.shape != (N, K) or Wq_up.shape != (N, K):
        raise ValueError("Wq_gate and Wq_up must both be [N, K] with Xq's K")
    if not (Xq.is_contiguous() and Wq_gate.is_contiguous() and Wq_up.is_contiguous()):
        raise ValueError("Xq, Wq_gate and Wq_up must be contiguous")
    _require_like(x_scale, "x_scale", torch.float32, M, Xq)
    _require_like(w_scale_gate, "w_scale_gate", torch.float32, N, Xq)
    _require_like(w_scale_up, "w_scale_up", torch.float32, N, Xq)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=Xq.device)
    _require_out(out, "out", torch.bfloat16, (M, N), Xq)
    st = lib().fp8_linear_swiglu(_ptr(Xq), _ptr(x_scale), _ptr(Wq_gate), _ptr(w_scale_gate), _ptr(Wq_up),
                                 _ptr(w_scale_up), M, N, K, _ptr(out), out.stride(0), _stream(Xq))
    _check(st, "fp8_linear_swiglu")
    return out


def fp8_linear_w8a16_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().fp8_linear_w8a16_workspace_size(M, N, K))


def fp8_linear_w8a16(X: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Weight-only FP8 for small M (<= 64): bf16 activations X [M, K] times the
    dequantized codes Wq [N, K] with per-channel scales w_scale [N], fp32 sums.
    -> Y bf16 [M, N].  `workspace`: a zero-filled uint8 device buffer of at
    least fp8_linear_w8a16_workspace_size bytes (allocated here when None)."""
    _require_cuda(X, "X", torch.bfloat16)
    _require_cuda(Wq, "Wq", torch.uint8)
    M, K = X.shape
    N = Wq.shape[0]
    if Wq.shape != (N, K) or not Wq.is_contiguous():
        raise ValueError("Wq must be a contiguous [N, K] tensor with X's K")
    if X.stride(1) != 1:
        raise ValueError("X rows must be contiguous")
    _require_like(w_scale, "w_scale", torch.float32, N, X)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _require_out(out, "out", torch.bfloat16, (M, N), X)
    wsb = fp8_linear_w8a16_workspace_size(M, N, K) if 0 < M <= 64 else 0
    if workspace is None and wsb:
        workspace = torch.zeros(wsb, dtype=torch.uint8, device=X.device)
    if workspace is not None:   # its size is checked by the library (FP8Q_ERR_INVALID_ARG)
        _require_like(workspace, "workspace", torch.uint8, 0, X)
    st = lib().fp8_linear_w8a16(_ptr(X), X.stride(0), _ptr(Wq), _ptr(w_scale), M, N, K, _ptr(out), out.stride(0),
                                _ptr(workspace) if workspace is not None else None,
                                workspace.numel() if workspace is not None else 0, _stream(X))
    _check(st, "fp8_linear_w8a16")
    return out


def fp8_quant_kv(kv: torch.Tensor, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """FP8 KV cache: one amax/448 scale per (token, head) of a K or V tensor.
    kv bf16 [T, H, 128] (head_dim 128, contiguous) -> (codes uint8 [T, H, 128], scales fp32 [T, H]).
    A head's 128 values are one 128-group of the [T, H*128] rows, so this is
    fp8_quant_act in BLOCK128 mode on that view."""
    if kv.dim() != 3 or kv.shape[2] != 128 or not kv.is_contiguous():
        raise ValueError("kv must be a contiguous [tokens, heads, 128] tensor")
    T, H, D = kv.shape
    if out is None:
        q = torch.empty((T, H, D), dtype=torch.uint8, device=kv.device)
        s = torch.empty((T, H), dtype=torch.float32, device=kv.device)
    else:
        q, s = out
    fp8_quant_act(kv.view(T, H * D), BLOCK128, out=(q.view(T, H * D), s.view(T, H)))
    return q, s


def fp8_linear_workspace_size(M: int, N: int, K: int, mode: int = CHANNEL_TOKEN) -> int:
    return int(lib().fp8_linear_workspace_size(M, N, K, int(mode)))


def fp8_linear(Xq: torch.Tensor, x_scale: torch.Tensor, Wq: torch.Tensor, w_scale: torch.Tensor,
               mode: int = CHANNEL_TOKEN, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y bf16 [M, N] = dequant(Xq) . dequant(Wq)^T.  Workspace (small-M path) is
    taken from torch's caching allocator, zero-filled, unless given; a given one
    must have been zero-filled before its first use (every call leaves it all zero)."""
    _require_cuda(Xq, "Xq", torch.uint8)
    _require_cuda(Wq, "Wq", torch.uint8)
    M, K = Xq.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K:
        raise ValueError("Xq and Wq disagree on K")
    if not (Xq.is_contiguous() and Wq.is_contiguous()):
        raise ValueError("Xq and Wq must be contiguous")
    _require_like(x_scale, "x_scale", torch.float32, _numel(scale_shape_act(M, K, mode)), Xq)
    _require_like(w_scale, "w_scale", torch.float32, _numel(scale_shape_weight(N, K, mode)), Xq)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=Xq.device)
    _require_out(out, "out", torch.bfloat16, (M, N), Xq)
    need = fp8_linear_workspace_size(M, N, K, mode)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=Xq.device)
    if workspace is not None:   # its size is checked by the library (FP8Q_ERR_INVALID_ARG)
        _require_like(workspace, "workspace", torch.uint8, 0, Xq)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().fp8_linear(_ptr(Xq), _ptr(x_scale), _ptr(Wq), _ptr(w_scale), M, N, K, int(mode),
                          _ptr(out), out.stride(0), _ptr(workspace), wbytes, _stream(Xq))
    _check(st, "fp8_linear")
    return out


# ------------------------------------------ rotary positions, 4-bit KV cache ---

ROPE_HALF, ROPE_INTERLEAVED, ROPE_INVERSE = 0, 1, 2
_ROPE_SCALINGS = {"linear": 1, "llama3": 2, "yarn": 3}


class _RopeScaling(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("original_max_position", ctypes.c_double)]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class _Binding:
    """csrc/binding.cpp, loaded at the first use: its functions check their operands as the functions below do, call
    the entry point and return its status, or return None where an operand is not as expected (the function below then
    says what is wrong, or takes care of a device that is not the current one)."""

    def __getattr__(self, name):
        lib()
        if not os.path.exists(BINDING_PATH):
            raise ImportError(f"_kv4_binding.so not built ({BINDING_PATH}); run "
                              "python -m fp8_w8a8_quantized_amax_b200.build")
        spec = importlib.util.spec_from_file_location("_kv4_binding", BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        for f in ("rope", "append", "read", "attention"):
            setattr(self, f, getattr(module, f))
        return getattr(module, name)


_binding = _Binding()


def _raw_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _current_device() -> int:
    return torch.cuda.current_device()


# The same values without a Stream object and a check for initialisation (the operands are CUDA tensors by then).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", _current_device)


def _call(dev: int, name: str, *args) -> None:
    """lib().<name>(*args, the current stream of device `dev`) with that device current; raises on an error status."""
    f = getattr(lib(), name)
    if dev == _current_device():
        st = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _raw_stream(dev))
    if st:
        raise FP8QError(st, name)


def _where(dev: int) -> str:
    return f" on cuda:{dev}" if dev >= 0 else ""


def _heads(t: torch.Tensor, name: str, dev: int, shape) -> Tuple[int, int]:
    """(token, head) strides of a bf16 tensor of `shape` [tokens, heads, head_dim] with contiguous elements on CUDA
    device `dev`; those of dimensions of size 1 as in a contiguous tensor."""
    if t.get_device() != dev or dev < 0 or t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be a bf16 CUDA tensor{_where(dev)}, got {t.dtype} on {t.device}")
    if len(shape) != 3 or t.shape != shape:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] = {tuple(shape)}, got {tuple(t.shape)}")
    T, H, D = shape
    a, b, c = t.stride()
    if c != 1 and D != 1:
        raise ValueError(f"{name} must have unit stride in the last dimension")
    return (a if T > 1 else H * D), (b if H > 1 else D)


def _list(t: torch.Tensor, name: str, dtype, numel: int, dev: int) -> int:
    """The address of a 1-D operand: contiguous, of exactly numel elements, on CUDA device `dev`."""
    if t.get_device() != dev or dev < 0 or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor{_where(dev)}, got {t.dtype} on {t.device}")
    if t.dim() != 1 or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {numel} elements")
    return t.data_ptr()


def _whole(n, name: str) -> int:
    """A whole number (numpy's too) that a C int64 holds: ctypes would drop the bits above."""
    n = operator.index(n)
    if not -2 ** 63 <= n < 2 ** 63:
        raise ValueError(f"{name} must fit in 64 bits, got {n}")
    return n


def fp8q_rope_frequencies(rot_dim: int, theta: float = 500000.0, scaling: Optional[dict] = None,
                          device="cuda") -> torch.Tensor:
    """The rot_dim / 2 rotary frequencies (fp64, radians per position) on `device`.
    scaling: None, or a dict with "type" ("linear", "llama3" or "yarn"), "factor", and for the latter two
    "original_max_position" and "low" / "high" (llama3: 1 / 4, yarn: 1 / 32 unless given)."""
    s = None
    if scaling is not None:
        kind = scaling.get("type")
        if kind not in _ROPE_SCALINGS:
            raise ValueError(f"unknown rope scaling {kind!r}")
        s = _RopeScaling(_ROPE_SCALINGS[kind], float(scaling["factor"]), float(scaling.get("low", 1.0)),
                         float(scaling.get("high", 32.0 if kind == "yarn" else 4.0)),
                         float(scaling.get("original_max_position", 0.0)))
    host = torch.empty(max(0, int(rot_dim)) // 2, dtype=torch.float64)
    st = lib().fp8q_rope_frequencies(host.data_ptr() or None, int(rot_dim), float(theta),
                                     ctypes.byref(s) if s is not None else None)
    _check(st, "fp8q_rope_frequencies")
    return host.to(device)


def fp8q_rope(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, interleaved: bool = False,
              inverse: bool = False, mscale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate bf16 heads x [T, H, D] by positions [T] (int64) times freq (fp64 [rot_dim / 2], from
    fp8q_rope_frequencies); elements from rot_dim on are copied.  `out` may be x itself, else must not overlap it."""
    flags = (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_INVERSE if inverse else 0)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    if _binding.rope(x, positions, freq, flags, float(mscale), out) == OK:
        return out
    dev, shape = x.get_device(), x.shape
    xt, xh = _heads(x, "x", dev, shape)
    T, H, D = shape
    pairs = freq.numel()
    at, f = _list(positions, "positions", torch.int64, T, dev), _list(freq, "freq", torch.float64, pairs, dev)
    yt, yh = (xt, xh) if out is x else _heads(out, "out", dev, shape)
    _call(dev, "fp8q_rope", x.data_ptr(), T, H, D, xt, xh, at, f, 2 * pairs, flags, float(mscale), out.data_ptr(),
          yt, yh)
    return out


def fp8q_kv4_page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of a KV4Cache's k_pages (or v_pages); 0 for sizes that are not supported."""
    return int(lib().fp8q_kv4_page_bytes(_whole(page_size, "page_size"), _whole(kv_heads, "kv_heads"),
                                         _whole(head_dim, "head_dim")))


class KV4Cache:
    """A paged KV cache of E2M1 codes with an E4M3 scale for each 16 elements (4.5 bits an element).

    k_pages, v_pages: uint8 CUDA tensors [num_pages, kv_heads, page_size * 9 * head_dim / 16], contiguous (KV4Cache.empty
    makes them).  k_scale, v_scale: the static fp32 factors of all values, amax / 2688 of a calibration set for the
    formats' whole range.  None of them can be changed afterwards."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, page_size: int, head_dim: int = 128,
                 k_scale: float = 1.0, v_scale: float = 1.0):
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if t.get_device() < 0 or t.get_device() != k_pages.get_device() or t.dtype != torch.uint8:
                raise ValueError(f"{name} must be a uint8 CUDA tensor (both on one device)")
            if t.dim() != 3 or not t.is_contiguous() or t.shape != k_pages.shape or \
                    t.shape[2] != page_size * (head_dim * 9 // 16):
                raise ValueError(f"{name} must be contiguous [num_pages, kv_heads, page_size * 9 * head_dim / 16]")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.num_pages, self.kv_heads = int(k_pages.shape[0]), int(k_pages.shape[1])
        self.page_size, self.head_dim = int(page_size), int(head_dim)
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.device, self._dev = k_pages.device, k_pages.get_device()
        self._struct = _CacheStruct(k_pages.data_ptr(), v_pages.data_ptr(), self.num_pages, self.page_size,
                                    self.kv_heads, self.head_dim, self.k_scale, self.v_scale)
        self._ref = ctypes.byref(self._struct)
        self._at = ctypes.addressof(self._struct)

    def __setattr__(self, name, value):              # the calls read what __init__ laid down for them
        if "_at" in self.__dict__:
            raise AttributeError(f"KV4Cache.{name} cannot be changed: make another cache over the same pages")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int = 64, head_dim: int = 128, k_scale: float = 1.0,
              v_scale: float = 1.0, device="cuda") -> "KV4Cache":
        """A cache of num_pages pages of page_size tokens, all zero."""
        shape = (num_pages, kv_heads, page_size * (head_dim * 9 // 16))
        return cls(torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros(shape, dtype=torch.uint8, device=device), page_size, head_dim, k_scale, v_scale)


def fp8q_kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    positions: Optional[torch.Tensor] = None, freq: Optional[torch.Tensor] = None,
                    interleaved: bool = False, mscale: float = 1.0) -> None:
    """Quantize k and v (bf16 [T, kv_heads, head_dim]) into the cache's slots ([T] int64, page * page_size + row;
    negative: skipped), k rotated by positions * freq on the way (as it is with both None)."""
    dev, flags = cache._dev, ROPE_INTERLEAVED if interleaved else 0
    if _binding.append(cache._at, dev, k, v, slots, positions, freq, flags, float(mscale)) == OK:
        return
    T = k.shape[0]
    shape = (T, cache.kv_heads, cache.head_dim)
    kt, kh = _heads(k, "k", dev, shape)
    vt, vh = _heads(v, "v", dev, shape)
    R, at, f = 0, None, None
    if positions is not None and freq is not None:
        pairs = freq.numel()
        R = 2 * pairs
        at, f = _list(positions, "positions", torch.int64, T, dev), _list(freq, "freq", torch.float64, pairs, dev)
    elif positions is not None or freq is not None:
        raise ValueError("positions and freq are given together")
    _call(dev, "fp8q_kv4_append", cache._ref, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
          _list(slots, "slots", torch.int64, T, dev), T, at, f, R, flags, float(mscale))


def fp8q_kv4_read(cache: KV4Cache, slots: torch.Tensor, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """The cached keys and values of slots [T] (int64) as bf16 [T, kv_heads, head_dim]; zeros for a negative slot."""
    dev, T = cache._dev, slots.numel()
    shape = (T, cache.kv_heads, cache.head_dim)
    k, v = torch.empty((2, *shape), dtype=torch.bfloat16, device=cache.device) if out is None else out
    if _binding.read(cache._at, dev, slots, k, v) == OK:
        return k, v
    at = _list(slots, "slots", torch.int64, T, dev)
    kt, kh = _heads(k, "k", dev, shape)
    vt, vh = _heads(v, "v", dev, shape)
    _call(dev, "fp8q_kv4_read", cache._ref, at, T, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh)
    return k, v


def fp8q_kv4_attention_workspace_size(cache: KV4Cache, num_seqs: int, tokens: int, q_heads: int,
                                      max_q_len: int = 1) -> int:
    sizes = (_whole(num_seqs, "num_seqs"), _whole(tokens, "tokens"), _whole(q_heads, "q_heads"), _whole(max_q_len, "max_q_len"))
    with torch.cuda.device(cache._dev):
        return int(lib().fp8q_kv4_attention_workspace_size(cache._ref, *sizes))


def fp8q_kv4_attention(q: torch.Tensor, cache: KV4Cache, page_table: torch.Tensor, kv_len: torch.Tensor,
                       q_start: Optional[torch.Tensor] = None, max_q_len: int = 1, sm_scale: Optional[float] = None,
                       causal: bool = True, window: int = 0, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of new tokens over the cache, which already holds them.

    q bf16 [T, q_heads, head_dim]; page_table int32 [B, max_pages]; kv_len int32 [B], tokens in the cache.
    q_start int32 [B + 1]: sequence b's rows of q are its last q_start[b + 1] - q_start[b] tokens, at most max_q_len
    (None: one row per sequence).  Rows behind the last sequence's are left as they were (in a new `out` they hold
    anything).  lse: fp32 [T, q_heads], written when given.  `workspace`: a uint8 buffer of
    fp8q_kv4_attention_workspace_size bytes, zero-filled before its first use and then kept from call to call (allocated
    here when None, which costs its zero-filling each time: up to 39 MB for many rows), not shared by calls in flight at
    once.  `out` must not overlap q.
    max_q_len chooses the kernel for the whole call: prompts and single tokens are faster in two calls.
    -> out bf16 [T, q_heads, head_dim]"""
    dev, shape = cache._dev, q.shape
    if sm_scale is None:
        sm_scale = cache.head_dim ** -0.5
    if out is not None and workspace is not None and \
            _binding.attention(cache._at, dev, q, page_table, kv_len, q_start, max_q_len, float(sm_scale), bool(causal),
                               window, out, lse, workspace) == OK:
        return out
    max_q_len, window, sm_scale = _whole(max_q_len, "max_q_len"), _whole(window, "window"), float(sm_scale)
    qt, qh = _heads(q, "q", dev, shape)
    T, Hq, D = shape
    if D != cache.head_dim:
        raise ValueError(f"q must have head_dim {cache.head_dim}")
    if page_table.dtype is not torch.int32 or page_table.get_device() != dev or page_table.dim() != 2:
        raise ValueError("page_table must be int32 [sequences, max_pages] on the cache's device")
    (B, max_pages), (row, unit) = page_table.shape, page_table.stride()
    if unit != 1 and max_pages > 1:
        raise ValueError("page_table's rows must be contiguous")
    lens = _list(kv_len, "kv_len", torch.int32, B, dev)
    starts = None if q_start is None else _list(q_start, "q_start", torch.int32, B + 1, dev)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    ot, oh = _heads(out, "out", dev, shape)
    sums = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.get_device() != dev or lse.shape != (T, Hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous fp32 {(T, Hq)} on the cache's device")
        sums = lse.data_ptr()
    if workspace is None:
        workspace = torch.zeros(fp8q_kv4_attention_workspace_size(cache, B, T, Hq, max_q_len), dtype=torch.uint8,
                                device=q.device)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the cache's device")
    _call(dev, "fp8q_kv4_attention", cache._ref, q.data_ptr(), qt, qh, T, Hq, page_table.data_ptr(),
          row if B > 1 else max_pages, max_pages, lens, starts, B, max_q_len, sm_scale,
          1 if causal else 0, window, out.data_ptr(), ot, oh, sums, workspace.data_ptr(), workspace.numel())
    return out                     # (the workspace's size is checked by the library: FP8Q_ERR_INVALID_ARG)


def device_error(clear: bool = True) -> int:
    """Device-side error word: nonzero after a kernel gave up waiting, or after the KV cache's calls met a slot past the
    cache (0x201), a page outside it (0x202) or bad lengths of a sequence (0x203)."""
    return int(lib().fp8q_device_error(1 if clear else 0))


def version() -> int:
    return int(lib().fp8q_version())


# Short aliases.
quant_weight = fp8_quant_weight
quant_act = fp8_quant_act
linear = fp8_linear
