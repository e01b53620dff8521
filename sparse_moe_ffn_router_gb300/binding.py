"""ctypes binding of the C ABI in include/moe.h (argument marshalling only).

Each function has the name of the C entry point it calls and takes torch CUDA tensors; it
passes their device pointers and the current CUDA stream, and raises MoEError when the
library returns a status other than MOE_OK. Nothing here computes any part of the layer.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from dataclasses import dataclass, fields

import torch

from . import build as _build

MOE_STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE", 3: "MOE_ERR_MISALIGNED",
              4: "MOE_ERR_WORKSPACE_TOO_SMALL", 5: "MOE_ERR_CUDA", 6: "MOE_ERR_TIMEOUT", 7: "MOE_ERR_DEVICE"}
EXPORTED = ["moe_workspace_size", "moe_workspace_init", "moe_route", "moe_forward", "moe_rmsnorm",
            "moe_last_device_error", "moe_workspace_tap", "moe_set_trace", "moe_launch_count", "moe_route_noalloc", "moe_status_string",
            "moe_router_stats", "moe_expert_shadow_size", "moe_forward_host_experts", "moe_forward_host_io",
            "moe_test_set_wait", "moe_w4_size", "moe_w4_quantize", "moe_w4_pack", "moe_w4_dequantize",
            "moe_w4_linear_workspace_size", "moe_w4_linear", "moe_forward_w4", "moe_w4_workspace_tap", "moe_sort_pairs",
            "moe_dispatch", "moe_dispatch_backward", "moe_combine", "moe_combine_backward", "moe_linear_workspace_size", "moe_linear",
            "moe_linear_backward", "moe_norm_workspace_size", "moe_norm_residual", "moe_norm_residual_backward"]
KERNELS = {"router_scores": 0, "router_topk": 1, "dispatch_local": 2, "dispatch_scan": 3, "dispatch_scatter": 4,
           "gate_up": 5, "down": 6, "combine": 7, "rmsnorm": 8, "shared_gate": 9, "gather": 10, "gemm_plan": 11,
           "decode_fused": 12, "router_stats": 13, "fetch_experts": 14,
           "copy_rows": 15, "w4_pack": 16, "w4_linear": 17,
           "w4_fused": 18, "sort_pairs": 19, "spread_rows": 20, "gather_rows": 21, "linear": 22, "linear_backward": 23,
           "norm": 24, "norm_backward": 25}


# moe_dims.flags: router and shared-gate scores rounded to bf16 before ranking and sigmoid
FLAG_BF16_SCORES = 1
# moe_test_set_wait: the signal held back so that a bounded device wait runs out
TEST_SUPPRESS_SCORE = 1
TEST_SUPPRESS_STAGE = 2


# moe_w4_format.format and the layout of a packed matrix
W4_INT4 = 0
W4_INT4_ZP = 1
W4_E2M1 = 2
W4_ROWS = 0
W4_GATE_UP = 1


class W4Format(ctypes.Structure):
    """moe_w4_format: the codes (W4_INT4, W4_INT4_ZP, W4_E2M1) and the columns to a scale (32, 64, 128)."""
    _fields_ = [("format", ctypes.c_int32), ("group", ctypes.c_int32)]


class Dims(ctypes.Structure):
    """moe_dims; a dims tuple is (T, H, E, K, I, Is) or (T, H, E, K, I, Is, flags)."""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("I", ctypes.c_int32), ("Is", ctypes.c_int32), ("flags", ctypes.c_int32)]


# moe_dtype, moe_act and moe_gate
BF16, FP16, FP32 = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_SIGMOID, ACT_SWIGLU = range(6)
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_FULL = range(4)
NORM_POST = 1
_TORCH = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32}
_DTYPE = {v: k for k, v in _TORCH.items()}


class _Dims(ctypes.Structure):
    """Sizes of a call, with what the checks of its tensors need worked out once (again after a field is set)."""

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        self.__dict__.pop("checked", None)

    def __getattr__(self, name):
        if name != "checked":
            raise AttributeError(name)
        c = self.__dict__["checked"] = self._checked()
        return c


class LinearDims(_Dims):
    """moe_linear_dims: T rows of K columns through one matrix [N, K], or through E of them by the rows' expert."""
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "N", "K", "E", "act", "dtype")]

    def __init__(self, T, N, K, E=1, act=ACT_NONE, dtype=BF16):
        super().__init__(int(T), int(N), int(K), int(E), int(act), int(dtype))

    def _checked(self):
        """Type, and the shapes of x, out, z, w, bias and offsets; the one matrix of E = 1 may come without its first dimension."""
        dt = _TORCH.get(self.dtype)
        if dt is None:
            raise MoEError(1, "moe_linear_dims")
        T, N, K, E = self.T, self.N, self.K, self.E
        return (dt, (T, K), (T, N // 2 if self.act == ACT_SWIGLU else N), (T, N), (E, N, K), (N, K) if E == 1 else None, (E, N),
                (N,) if E == 1 else None, (E + 1,))


class NormDims(_Dims):
    """moe_norm_dims: T rows of H columns; gate: GATE_*, gate_act: ACT_NONE, ACT_SIGMOID or ACT_SILU of it."""
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "dtype", "gate", "gate_act", "flags")] + [
        (n, ctypes.c_float) for n in ("eps", "branch_scale", "residual_scale")]

    def __init__(self, T, H, dtype=BF16, post=True, gate=GATE_NONE, gate_act=ACT_NONE, eps=1e-6, branch_scale=1.0, residual_scale=1.0):
        super().__init__(int(T), int(H), int(dtype), int(gate), int(gate_act), NORM_POST if post else 0, float(eps), float(branch_scale),
                         float(residual_scale))

    def _checked(self):
        """Type, and the shapes of rows, gammas and gate."""
        dt, T, H = _TORCH.get(self.dtype), self.T, self.H
        if dt is None:
            raise MoEError(1, "moe_norm_dims")
        return dt, (T, H), (H,), {GATE_TOKEN: (T,), GATE_CHANNEL: (H,), GATE_FULL: (T, H)}.get(self.gate, ())


class CWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("router_w", "router_b", "gate_up", "down", "shared_gate_up",
                                                "shared_down", "shared_gate")]


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_status_string(status)}")


@dataclass
class Weights:
    """One layer's weights (bf16 CUDA tensors, [Out, In] row-major); router_b may be None."""
    router_w: torch.Tensor
    router_b: torch.Tensor | None
    gate_up: torch.Tensor
    down: torch.Tensor
    shared_gate_up: torch.Tensor
    shared_down: torch.Tensor
    shared_gate: torch.Tensor

    @classmethod
    def from_dict(cls, d: dict) -> "Weights":
        return cls(**{f.name: d.get(f.name) for f in fields(cls)})

    def to_c(self) -> CWeights:
        return CWeights(_ptr(self.router_w), _ptr(self.router_b), _ptr(self.gate_up), _ptr(self.down),
                        _ptr(self.shared_gate_up), _ptr(self.shared_down), _ptr(self.shared_gate))


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load_library(build_if_missing: bool = True):
    """Load libmoe_gb300.so (building it first when it is absent or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if build_if_missing:
                _build.build()
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"CUDA library {_build.LIB} is missing; run build() first")
            lib = ctypes.CDLL(_build.LIB)
            P, S = ctypes.c_void_p, ctypes.c_size_t
            D, W = ctypes.POINTER(Dims), ctypes.POINTER(CWeights)
            st = ctypes.c_int
            lib.moe_workspace_size.restype = S
            lib.moe_workspace_size.argtypes = [D]
            lib.moe_workspace_init.restype = st
            lib.moe_workspace_init.argtypes = [P, S, P]
            lib.moe_route.restype = st
            lib.moe_route.argtypes = [D, P, W, P, P, P, P, P, P, S, P]
            lib.moe_forward.restype = st
            lib.moe_forward.argtypes = [D, P, W, P, P, P, S, P]
            lib.moe_rmsnorm.restype = st
            lib.moe_rmsnorm.argtypes = [D, P, P, ctypes.c_float, P, P]
            lib.moe_last_device_error.restype = st
            lib.moe_last_device_error.argtypes = [P, P]
            lib.moe_workspace_tap.restype = st
            lib.moe_workspace_tap.argtypes = [D, ctypes.c_int, ctypes.POINTER(S), ctypes.POINTER(S)]
            lib.moe_w4_workspace_tap.restype = st
            lib.moe_w4_workspace_tap.argtypes = [D, ctypes.c_int, ctypes.POINTER(S), ctypes.POINTER(S)]
            lib.moe_set_trace.restype = st
            lib.moe_set_trace.argtypes = [ctypes.c_int, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.c_int]
            lib.moe_launch_count.restype = ctypes.c_uint64
            lib.moe_launch_count.argtypes = []
            lib.moe_route_noalloc.restype = st
            lib.moe_route_noalloc.argtypes = [D, P, W, P, P, P, P, P, P]
            lib.moe_router_stats.restype = st
            lib.moe_router_stats.argtypes = [D, P, W, P, P, P, P, S, P]
            lib.moe_expert_shadow_size.restype = S
            lib.moe_expert_shadow_size.argtypes = [D]
            lib.moe_forward_host_experts.restype = st
            lib.moe_forward_host_experts.argtypes = [D, P, W, P, P, P, S, P, S, P]
            lib.moe_forward_host_io.restype = st
            lib.moe_forward_host_io.argtypes = [D, P, W, P, P, P, P, P, S, P]
            F, I32 = ctypes.POINTER(W4Format), ctypes.c_int32
            lib.moe_w4_size.restype = S
            lib.moe_w4_size.argtypes = [F, I32, I32, I32]
            lib.moe_w4_quantize.restype = st
            lib.moe_w4_quantize.argtypes = [F, I32, I32, I32, I32, P, P, S, P]
            lib.moe_w4_pack.restype = st
            lib.moe_w4_pack.argtypes = [F, I32, I32, I32, I32, P, P, P, P, S, P]
            lib.moe_w4_dequantize.restype = st
            lib.moe_w4_dequantize.argtypes = [F, I32, I32, I32, I32, P, S, P, P]
            lib.moe_w4_linear_workspace_size.restype = S
            lib.moe_w4_linear_workspace_size.argtypes = [F, I32, I32, I32]
            lib.moe_w4_linear.restype = st
            lib.moe_w4_linear.argtypes = [F, I32, I32, I32, P, P, S, P, P, P, S, P]
            lib.moe_forward_w4.restype = st
            lib.moe_forward_w4.argtypes = [D, F, P, W, P, P, P, S, P]
            L, N = ctypes.POINTER(LinearDims), ctypes.POINTER(NormDims)
            lib.moe_sort_pairs.restype = st
            lib.moe_sort_pairs.argtypes = [I32, I32, I32, P, P, P, P, P, P]
            for name in ("moe_dispatch", "moe_combine"):
                getattr(lib, name).restype = st
            lib.moe_dispatch.argtypes = [I32, I32, I32, I32, P, P, P, P, P]
            lib.moe_combine.argtypes = [I32, I32, I32, I32, P, P, P, P, P, P]
            for name in ("moe_dispatch_backward", "moe_combine_backward"):
                getattr(lib, name).restype = st
                getattr(lib, name).argtypes = [I32, I32, I32, I32, P, P, P, P, P, P, P]
            lib.moe_linear_workspace_size.restype = S
            lib.moe_linear_workspace_size.argtypes = [L, I32]
            lib.moe_linear.restype = st
            lib.moe_linear.argtypes = [L, P, P, P, P, P, P, P, P, S, P]
            lib.moe_linear_backward.restype = st
            lib.moe_linear_backward.argtypes = [L, P, P, P, P, P, P, P, P, P, S, P]
            lib.moe_norm_workspace_size.restype = S
            lib.moe_norm_workspace_size.argtypes = [N]
            lib.moe_norm_residual.restype = st
            lib.moe_norm_residual.argtypes = [N, P, P, P, P, P, P, P, P]
            lib.moe_norm_residual_backward.restype = st
            lib.moe_norm_residual_backward.argtypes = [N, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P]
            lib.moe_test_set_wait.restype = st
            lib.moe_test_set_wait.argtypes = [ctypes.c_uint64, ctypes.c_int]
            lib.moe_status_string.restype = ctypes.c_char_p
            lib.moe_status_string.argtypes = [ctypes.c_int]
            _lib = lib
    return _lib


def _status_string(s: int) -> str:
    try:
        return load_library(build_if_missing=False).moe_status_string(s).decode()
    except Exception:  # the library itself may be what is missing
        return MOE_STATUS.get(s, f"status {s}")


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("the MoE layer runs on the GPU only: pass CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# The current stream's handle without building a torch.cuda.Stream object (2.9 us on the GB300 host
# against 0.1 us), where this torch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dims(d) -> Dims:
    return d if isinstance(d, Dims) else Dims(*[int(v) for v in d])


def _check(status: int, what: str):
    if status != 0:
        raise MoEError(status, what)


def moe_workspace_size(dims) -> int:
    return int(load_library().moe_workspace_size(ctypes.byref(_dims(dims))))


def moe_workspace_init(workspace: torch.Tensor, stream=None):
    _check(load_library().moe_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                             _stream(stream)), "moe_workspace_init")


def new_workspace(dims, device="cuda") -> torch.Tensor:
    """A zero-filled uint8 device workspace of moe_workspace_size(dims) bytes."""
    n = moe_workspace_size(dims)
    if n == 0:
        raise MoEError(2, "moe_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_route(dims, x, weights: Weights, ids, topk_w, counts, offsets, perm, workspace, stream=None):
    w = weights.to_c()
    _check(load_library().moe_route(ctypes.byref(_dims(dims)), _ptr(x), ctypes.byref(w), _ptr(ids), _ptr(topk_w),
                                    _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)), "moe_route")


def moe_route_noalloc(dims, x, weights: Weights, ids, topk_w, counts, offsets, perm, stream=None):
    """moe_route without a workspace (for callers that cannot allocate device memory)."""
    w = weights.to_c()
    _check(load_library().moe_route_noalloc(ctypes.byref(_dims(dims)), _ptr(x), ctypes.byref(w), _ptr(ids),
                                            _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(perm), _stream(stream)),
           "moe_route_noalloc")


def moe_router_stats(dims, x, weights: Weights, P, f, loss, workspace, stream=None):
    """Load-balancing statistics: P [E] and f [E] fp32 (mean router probability, share of the
    assignments) and loss [1] fp32 = 0.001 * E * sum(f * P)."""
    w = weights.to_c()
    _check(load_library().moe_router_stats(ctypes.byref(_dims(dims)), _ptr(x), ctypes.byref(w), _ptr(P), _ptr(f),
                                           _ptr(loss), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                           _stream(stream)), "moe_router_stats")


def moe_forward(dims, x, weights: Weights, residual, out, workspace, stream=None):
    w = weights.to_c()
    _check(load_library().moe_forward(ctypes.byref(_dims(dims)), _ptr(x), ctypes.byref(w), _ptr(residual), _ptr(out),
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(stream)), "moe_forward")


def _ptr_host(t) -> int:
    """Address of a pinned (page-locked) host tensor, for the host-resident expert weights."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if t.is_cuda or not t.is_pinned():
        raise ValueError("host-resident expert weights must be pinned CPU tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def moe_expert_shadow_size(dims) -> int:
    return int(load_library().moe_expert_shadow_size(ctypes.byref(_dims(dims))))


def moe_forward_host_experts(dims, x, weights: Weights, residual, out, shadow, workspace, stream=None):
    """moe_forward with weights.gate_up and weights.down in pinned host memory: the experts
    each call touches are copied over the host link into `shadow` (a uint8 CUDA tensor of
    moe_expert_shadow_size(dims) bytes) and run from there."""
    w = CWeights(*[(_ptr_host(getattr(weights, f.name)) if f.name in ("gate_up", "down") else _ptr(getattr(weights, f.name)))
                   for f in fields(weights)])
    _check(load_library().moe_forward_host_experts(ctypes.byref(_dims(dims)), _ptr(x), ctypes.byref(w), _ptr(residual),
                                                   _ptr(out), _ptr(shadow), shadow.numel() * shadow.element_size(),
                                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                   _stream(stream)), "moe_forward_host_experts")


def _ptr_cpu(t, nbytes: int) -> int | None:
    """Address of a contiguous CPU tensor (pinned or pageable) of at least nbytes bytes."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if t.is_cuda:
        raise ValueError("host-side token rows must be CPU tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"host tensor holds {t.numel() * t.element_size()} bytes, the layer needs {nbytes}")
    return t.data_ptr()


def moe_forward_host_io(dims, x, weights: Weights, residual, out, x_dev, out_dev, workspace, stream=None):
    """moe_forward with the token rows in host memory: x (and residual, when given) are CPU
    tensors copied into the device staging tensors x_dev (and out_dev), the layer runs, and
    out_dev is copied back into the CPU tensor out, all in order on `stream`. Pinned host
    tensors keep the copies asynchronous (and one token, with x, residual and out pinned, runs
    in one kernel that reads and writes them over the host link, with no copy); out holds the
    result once the stream has passed the call."""
    d = _dims(dims)
    nbytes = d.T * d.H * 2
    for t in (x_dev, out_dev):
        if t is not None and t.numel() * t.element_size() < nbytes:
            raise ValueError("device staging tensors must hold [T, H] bf16")
    _check(load_library().moe_forward_host_io(ctypes.byref(d), _ptr_cpu(x, nbytes), ctypes.byref(weights.to_c()),
                                              _ptr_cpu(residual, nbytes), _ptr_cpu(out, nbytes), _ptr(x_dev),
                                              _ptr(out_dev), _ptr(workspace),
                                              workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_forward_host_io")


class ForwardHostIO:
    """moe_forward_host_io with everything but the host buffers marshalled once.

    A decode loop calls the same layer with the same weights, staging tensors and workspace
    on every step; this object converts those (and the stream, the current one when none is
    given) into C arguments at construction and keeps references to the tensors, so each
    call only checks and passes the host tensors. The tensors must not be resized or
    re-pointed (``set_``) while the object is in use."""

    def __init__(self, dims, weights: Weights, x_dev, out_dev, workspace, stream=None):
        self._d = _dims(dims)
        self._nbytes = self._d.T * self._d.H * 2
        for t in (x_dev, out_dev):
            if t is not None and t.numel() * t.element_size() < self._nbytes:
                raise ValueError("device staging tensors must hold [T, H] bf16")
        self._w = weights.to_c()
        self._keep = (weights, x_dev, out_dev, workspace)
        self._fixed = (ctypes.byref(self._d), ctypes.byref(self._w))
        self._staging = (_ptr(x_dev), _ptr(out_dev), _ptr(workspace), workspace.numel() * workspace.element_size(),
                         _stream(stream))
        self._fn = load_library().moe_forward_host_io

    def __call__(self, x, out, residual=None):
        n = self._nbytes
        _check(self._fn(self._fixed[0], _ptr_cpu(x, n), self._fixed[1], _ptr_cpu(residual, n), _ptr_cpu(out, n),
                        *self._staging), "moe_forward_host_io")


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def moe_w4_size(fmt: W4Format, rows: int, cols: int, n: int = 1) -> int:
    """Bytes of n packed 4-bit matrices [rows, cols] (0 when the format or shape is not supported)."""
    return int(load_library().moe_w4_size(ctypes.byref(fmt), int(n), int(rows), int(cols)))


@functools.lru_cache(maxsize=1024)
def _w4_bytes(fmt: int, group: int, rows: int, cols: int) -> int:
    return moe_w4_size(W4Format(fmt, group), rows, cols)


def new_w4(fmt: W4Format, rows: int, cols: int, n: int = 1, device="cuda") -> torch.Tensor:
    """An uninitialised uint8 CUDA tensor [n, bytes of one packed matrix]."""
    b = _w4_bytes(fmt.format, fmt.group, int(rows), int(cols))
    if b == 0 or n < 0:
        raise MoEError(2, "moe_w4_size")
    return torch.empty(int(n), b, dtype=torch.uint8, device=device)


def _matrices(t) -> tuple[int, int, int]:
    if t.dim() not in (2, 3):
        raise ValueError("weights are [rows, cols] or [n, rows, cols]")
    return (1, *t.shape) if t.dim() == 2 else tuple(t.shape)


def _device(t, dtype=None, what: str = "") -> int:
    """The current CUDA device, where the kernels will run; t: the first tensor of the call."""
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        _ptr(t)
    return torch.cuda.current_device()


def _here(device: int, *tensors) -> list:
    """_ptr of each tensor; all must be on the given device."""
    try:
        ptrs = [None if t is None else t.data_ptr() if t.get_device() == device and t.is_contiguous() else -1 for t in tensors]
    except AttributeError:
        raise TypeError("expected a torch.Tensor") from None
    if -1 in ptrs:
        _ptr(tensors[ptrs.index(-1)])
        raise ValueError(f"tensors must be on the current CUDA device ({device})")
    return ptrs


def _stream_of(stream, device: int) -> int:
    return _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)


def moe_w4_quantize(fmt: W4Format, w, packed, layout: int = W4_ROWS, stream=None):
    """packed = the 4-bit form of the bf16 weights w [rows, cols] or [n, rows, cols]."""
    n, rows, cols = _matrices(w)
    dev = _device(w, torch.bfloat16, "w")
    src, dst = _here(dev, w, packed)
    _check(load_library().moe_w4_quantize(ctypes.byref(fmt), n, rows, cols, int(layout), src, dst, _nbytes(packed),
                                          _stream_of(stream, dev)), "moe_w4_quantize")


def moe_w4_pack(fmt: W4Format, codes, scales, zeros, packed, layout: int = W4_ROWS, stream=None):
    """packed = a checkpoint's codes [.., rows, cols / 2] uint8 (even column in the low nibble), scales
    [.., rows, cols / group] bf16 and zero points [.., rows, cols / group] uint8 (or None)."""
    n, rows, half = _matrices(codes)
    groups = (*codes.shape[:-1], 2 * half // fmt.group if fmt.group > 0 else 0)
    if codes.dtype != torch.uint8 or (zeros is not None and zeros.dtype != torch.uint8):
        raise TypeError("codes and zeros must be uint8")
    if tuple(scales.shape) != groups or (zeros is not None and tuple(zeros.shape) != groups):
        raise ValueError(f"scales and zeros must be {list(groups)}")
    dev = _device(scales, torch.bfloat16, "scales")
    c, s, z, dst = _here(dev, codes, scales, zeros, packed)
    _check(load_library().moe_w4_pack(ctypes.byref(fmt), n, rows, 2 * half, int(layout), c, s, z, dst, _nbytes(packed),
                                      _stream_of(stream, dev)), "moe_w4_pack")


def moe_w4_dequantize(fmt: W4Format, packed, w, layout: int = W4_ROWS, stream=None):
    """w [rows, cols] or [n, rows, cols] = the bf16 weights the packed form stands for."""
    n, rows, cols = _matrices(w)
    dev = _device(w, torch.bfloat16, "w")
    src, dst = _here(dev, packed, w)
    _check(load_library().moe_w4_dequantize(ctypes.byref(fmt), n, rows, cols, int(layout), src, _nbytes(packed), dst,
                                            _stream_of(stream, dev)), "moe_w4_dequantize")


def new_w4_linear_workspace(fmt: W4Format, T: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A zero-filled uint8 device workspace for moe_w4_linear at these sizes."""
    n = int(load_library().moe_w4_linear_workspace_size(ctypes.byref(fmt), int(T), int(N), int(K)))
    if n == 0:
        raise MoEError(2, "moe_w4_linear_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_w4_linear(fmt: W4Format, x, packed, bias, out, workspace, stream=None):
    """out [T, N] = x [T, K] . W^T + bias, with W [N, K] packed (layout W4_ROWS)."""
    xs, os = x.shape, out.shape
    if len(xs) != 2 or len(os) != 2 or xs[0] != os[0]:
        raise ValueError("x is [T, K] and out [T, N]")
    T, K = xs
    N = os[1]
    if bias is not None and (bias.dtype != torch.bfloat16 or tuple(bias.shape) != (N,)):
        raise (TypeError if bias.dtype != torch.bfloat16 else ValueError)(f"bias must be bfloat16 [{N}]")
    if out.dtype != torch.bfloat16:
        raise TypeError(f"out must be {torch.bfloat16}, got {out.dtype}")
    dev = _device(x, torch.bfloat16, "x")
    px, pw, pb, po, ws = _here(dev, x, packed, bias, out, workspace)
    _check(load_library().moe_w4_linear(ctypes.byref(fmt), T, N, K, px, pw, _nbytes(packed), pb, po, ws, _nbytes(workspace),
                                        _stream_of(stream, dev)), "moe_w4_linear")


@functools.lru_cache(maxsize=256)
def _w4_layer(dims: tuple, fmt: int, group: int):
    """The dims (whole numbers) as passed to C, the bytes of the layer's packed gate_up, down, shared_gate_up and shared_down, and
    the elements of its bf16 tensors."""
    d = Dims(*dims)
    record = 1024 + 16 * (128 // group) * (3 if fmt == W4_INT4_ZP else 2) if group in (32, 64, 128) else 0
    h = (d.H + 127) // 128
    return d, (d.E * ((2 * d.I + 15) // 16) * h * record, d.E * ((d.H + 15) // 16) * ((d.I + 127) // 128) * record,
               ((2 * d.Is + 15) // 16) * h * record, ((d.H + 15) // 16) * ((d.Is + 127) // 128) * record), \
        (d.T * d.H, d.T * d.H, d.T * d.H, d.E * d.H, d.E, d.H)


_BF16, _U8 = torch.bfloat16, torch.uint8


def _w4_refuse(packed, needs, plain, counts):
    """Raises what is wrong with the tensors of moe_forward_w4."""
    for t, need in zip(packed, needs):
        if t is None or t.dtype != _U8:
            raise TypeError("the experts' weights must be packed 4-bit weights (uint8)")
        if t.numel() < need:
            raise ValueError(f"packed weights of {t.numel()} bytes, the layer's dims need {need}")
    for name, t, need in zip(("x", "out", "residual", "router_w", "router_b", "shared_gate"), plain, counts):
        if t is None:
            if name in ("residual", "router_b"):
                continue
            raise TypeError(f"{name} is missing")
        if t.dtype != _BF16:
            raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
        if t.numel() < need:
            raise ValueError(f"{name} holds {t.numel()} elements, the layer's dims need {need}")
    raise TypeError("expected torch.Tensors")


def moe_forward_w4(dims, fmt: W4Format, x, weights: Weights, residual, out, workspace, stream=None):
    """moe_forward with weights.gate_up, down, shared_gate_up and shared_down in packed 4-bit form
    (uint8 tensors of moe_w4_size bytes; gate_up layouts W4_GATE_UP, down layouts W4_ROWS)."""
    if isinstance(dims, Dims):
        dims = tuple(getattr(dims, f) for f, _ in Dims._fields_)
    d, needs, counts = _w4_layer(tuple(map(int, dims)), fmt.format, fmt.group)
    rw, rb, gu, dn, sgu, sdn, sg = (weights.router_w, weights.router_b, weights.gate_up, weights.down, weights.shared_gate_up,
                                    weights.shared_down, weights.shared_gate)
    rows, er, eb, hs = counts[0], counts[3], counts[4], counts[5]
    try:
        fits = (gu.dtype is dn.dtype is sgu.dtype is sdn.dtype is _U8 and x.dtype is out.dtype is rw.dtype is sg.dtype is _BF16
                and gu.numel() >= needs[0] and dn.numel() >= needs[1] and sgu.numel() >= needs[2] and sdn.numel() >= needs[3]
                and x.numel() >= rows and out.numel() >= rows and rw.numel() >= er and sg.numel() >= hs
                and (residual is None or residual.dtype is _BF16 and residual.numel() >= rows)
                and (rb is None or rb.dtype is _BF16 and rb.numel() >= eb))
    except AttributeError:
        fits = False
    if not fits:
        _w4_refuse((gu, dn, sgu, sdn), needs, (x, out, residual, rw, rb, sg), counts)
    dev = _device(x)
    px, po, res, router_w, router_b, gate, ws, *packed = _here(dev, x, out, residual, rw, rb, sg, workspace, gu, dn, sgu, sdn)
    w = CWeights(router_w, router_b, *packed, gate)
    _check(load_library().moe_forward_w4(ctypes.byref(d), ctypes.byref(fmt), px, ctypes.byref(w), res, po, ws, _nbytes(workspace),
                                         _stream_of(stream, dev)), "moe_forward_w4")


def _refuse(name: str, t, dtype, shapes, device: int):
    """Raises what is wrong with an argument that _ptr_of does not take."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape not in shapes:
        raise ValueError(f"{name} must be {' or '.join(str(list(s)) for s in shapes)}, got {list(t.shape)}")
    _ptr(t)
    raise ValueError(f"{name} must be on the current CUDA device ({device}), got {t.device}")


def _ptr_of(device: int, dtype, shape: tuple, name: str, t, other: tuple | None = None):
    """Address of an argument (None: none) once its type, shape (or other), layout and device are checked."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and (t.shape == shape or t.shape == other) and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, dtype, (shape,) if other is None else (shape, other), device)


_I32, _F32 = torch.int32, torch.float32


def moe_sort_pairs(E: int, ids, counts, offsets, perm, inv, stream=None):
    """Dispatch of the expert ids [T, K] int32: counts [E], offsets [E + 1], perm [T * K] (pairs t * K + k by expert,
    -1 behind the last) and inv [T * K] (each pair's place, -1 for an id outside [0, E))."""
    dev = _current("ids", ids)
    if ids.dim() != 2:
        raise ValueError("ids must be int32 [T, K]")
    shape = ids.shape
    T, K = shape
    flat = (T * K,)
    _check(load_library().moe_sort_pairs(T, K, E, _ptr_of(dev, _I32, shape, "ids", ids), _ptr_of(dev, _I32, (E,), "counts", counts),
                                         _ptr_of(dev, _I32, (E + 1,), "offsets", offsets), _ptr_of(dev, _I32, flat, "perm", perm, shape),
                                         _ptr_of(dev, _I32, flat, "inv", inv, shape), _stream_of(stream, dev)), "moe_sort_pairs")


def _exchange(token, rows, *pairs):
    """Device, type, T, K and H of a call on token rows [T, H] and experts' rows [T * K, H]; pairs: the call's tensors [T, K] (or flat,
    or None), which tell K where there are no tokens."""
    dev = _current("token rows", token)
    if not isinstance(rows, torch.Tensor):
        raise TypeError(f"experts' rows: expected a torch.Tensor, got {type(rows).__name__}")
    if token.dim() != 2 or rows.dim() != 2:
        raise ValueError("token rows are [T, H], experts' rows [T * K, H]")
    T, H = token.shape
    n = rows.shape[0]
    K = n // T if T else next((p.shape[1] for p in pairs if isinstance(p, torch.Tensor) and p.dim() == 2), 1)
    if n != T * K:
        raise ValueError(f"experts' rows must be T * K, T = {T}: got {n}")
    code = _DTYPE.get(token.dtype)
    if code is None:
        raise TypeError(f"token rows must be bfloat16, float16 or float32, got {token.dtype}")
    return dev, token.dtype, code, T, K, H


def moe_dispatch(x, inv, topk_w, rows, stream=None):
    """rows [T * K, H]: rows[inv[t, k]] = topk_w[t, k] * x[t] (topk_w None: the rows as they are)."""
    dev, dt, code, T, K, H = _exchange(x, rows, inv, topk_w)
    n = T * K
    _check(load_library().moe_dispatch(code, T, K, H, _ptr_of(dev, dt, (T, H), "x", x), _ptr_of(dev, _I32, (n,), "inv", inv, (T, K)),
                                       _ptr_of(dev, _F32, (T, K), "topk_w", topk_w, (n,)), _ptr_of(dev, dt, (n, H), "rows", rows),
                                       _stream_of(stream, dev)), "moe_dispatch")


def moe_dispatch_backward(drows, inv, topk_w, x, dx, dtopk_w=None, stream=None):
    """dx [T, H] = sum_k topk_w[t, k] * drows[inv[t, k]]; dtopk_w [T, K] (optional; x is read for it) = x[t] . drows[inv[t, k]]."""
    dev, dt, code, T, K, H = _exchange(dx, drows, inv, topk_w, dtopk_w)
    n = T * K
    _check(load_library().moe_dispatch_backward(code, T, K, H, _ptr_of(dev, dt, (n, H), "drows", drows), _ptr_of(dev, _I32, (n,), "inv", inv, (T, K)),
                                                _ptr_of(dev, _F32, (T, K), "topk_w", topk_w, (n,)), _ptr_of(dev, dt, (T, H), "x", x),
                                                _ptr_of(dev, dt, (T, H), "dx", dx), _ptr_of(dev, _F32, (T, K), "dtopk_w", dtopk_w, (n,)),
                                                _stream_of(stream, dev)), "moe_dispatch_backward")


def moe_combine(rows, inv, topk_w, residual, out, stream=None):
    """out [T, H] = residual + sum_k topk_w[t, k] * rows[inv[t, k]] (topk_w and residual may be None)."""
    dev, dt, code, T, K, H = _exchange(out, rows, inv, topk_w)
    n = T * K
    _check(load_library().moe_combine(code, T, K, H, _ptr_of(dev, dt, (n, H), "rows", rows), _ptr_of(dev, _I32, (n,), "inv", inv, (T, K)),
                                      _ptr_of(dev, _F32, (T, K), "topk_w", topk_w, (n,)), _ptr_of(dev, dt, (T, H), "residual", residual),
                                      _ptr_of(dev, dt, (T, H), "out", out), _stream_of(stream, dev)), "moe_combine")


def moe_combine_backward(dout, inv, topk_w, rows, drows, dtopk_w=None, stream=None):
    """drows[inv[t, k]] = topk_w[t, k] * dout[t]; dtopk_w [T, K] (optional; rows are read for it) = dout[t] . rows[inv[t, k]]."""
    dev, dt, code, T, K, H = _exchange(dout, drows, inv, topk_w, dtopk_w)
    n = T * K
    _check(load_library().moe_combine_backward(code, T, K, H, _ptr_of(dev, dt, (T, H), "dout", dout), _ptr_of(dev, _I32, (n,), "inv", inv, (T, K)),
                                               _ptr_of(dev, _F32, (T, K), "topk_w", topk_w, (n,)), _ptr_of(dev, dt, (n, H), "rows", rows),
                                               _ptr_of(dev, dt, (n, H), "drows", drows), _ptr_of(dev, _F32, (T, K), "dtopk_w", dtopk_w, (n,)),
                                               _stream_of(stream, dev)), "moe_combine_backward")


def new_linear_workspace(dims: LinearDims, backward: bool = False, device="cuda") -> torch.Tensor:
    """A zero-filled uint8 device workspace for moe_linear, or for moe_linear_backward, at these sizes."""
    n = int(load_library().moe_linear_workspace_size(ctypes.byref(dims), int(backward)))
    if n == 0:
        raise MoEError(2, "moe_linear_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _current(name: str, t) -> int:
    """The current CUDA device, where the kernels will run; t: the first tensor of the call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    return torch.cuda.current_device() if t.is_cuda else -2


def _sizes(dims, kind):
    """What the checks of a call's tensors go by, of dims of its kind."""
    if not isinstance(dims, kind):
        raise TypeError(f"dims: expected {kind.__name__}, got {type(dims).__name__}")
    return dims.checked


def _workspace(device: int, t):
    if t is not None and not isinstance(t, torch.Tensor):
        raise TypeError(f"workspace: expected a torch.Tensor, got {type(t).__name__}")
    if t is None or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on the current CUDA device ({device})")
    return t.data_ptr(), t.numel() * t.element_size()


def moe_linear(dims: LinearDims, x, w, bias, offsets, residual, out, z, workspace, stream=None):
    """out = act(x . W_e^T + bias_e) + residual, e the expert whose rows [offsets[e], offsets[e + 1]) hold x's row
    (offsets None: the one matrix); z (or None) receives the pre-activations for moe_linear_backward."""
    dt, rows, wide, pre, mat, mat1, vec, vec1, ends = _sizes(dims, LinearDims)
    dev = _current("x", x)
    _check(load_library().moe_linear(ctypes.byref(dims), _ptr_of(dev, dt, rows, "x", x), _ptr_of(dev, dt, mat, "w", w, mat1),
                                     _ptr_of(dev, dt, vec, "bias", bias, vec1), _ptr_of(dev, _I32, ends, "offsets", offsets),
                                     _ptr_of(dev, dt, wide, "residual", residual), _ptr_of(dev, dt, wide, "out", out),
                                     _ptr_of(dev, dt, pre, "z", z), *_workspace(dev, workspace), _stream_of(stream, dev)), "moe_linear")


def moe_linear_backward(dims: LinearDims, x, w, offsets, z, dout, dx, dw, dbias, workspace, stream=None):
    """Gradients of moe_linear's x, w and bias (each may be None) for the gradient dout of its result; the residual's is dout."""
    dt, rows, wide, pre, mat, mat1, vec, vec1, ends = _sizes(dims, LinearDims)
    dev = _current("dout", dout)
    _check(load_library().moe_linear_backward(
        ctypes.byref(dims), _ptr_of(dev, dt, rows, "x", x), _ptr_of(dev, dt, mat, "w", w, mat1), _ptr_of(dev, _I32, ends, "offsets", offsets),
        _ptr_of(dev, dt, pre, "z", z), _ptr_of(dev, dt, wide, "dout", dout), _ptr_of(dev, dt, rows, "dx", dx),
        _ptr_of(dev, dt, mat, "dw", dw, mat1), _ptr_of(dev, dt, vec, "dbias", dbias, vec1), *_workspace(dev, workspace),
        _stream_of(stream, dev)), "moe_linear_backward")


def new_norm_workspace(dims: NormDims, device="cuda") -> torch.Tensor:
    """A uint8 device workspace for moe_norm_residual_backward at these sizes."""
    n = int(load_library().moe_norm_workspace_size(ctypes.byref(dims)))
    if n == 0:
        raise MoEError(2, "moe_norm_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_norm_residual(dims: NormDims, y, residual, gate, gamma_post, gamma_pre, s, xn, stream=None):
    """s = residual_scale * residual + branch_scale * act(gate) * N(y; gamma_post), xn = N(s; gamma_pre); residual, the
    gammas and either result may be None, and N(y) is y for dims without post."""
    dt, rows, cols, gs = _sizes(dims, NormDims)
    dev = _current("y", y)
    _check(load_library().moe_norm_residual(
        ctypes.byref(dims), _ptr_of(dev, dt, rows, "y", y), _ptr_of(dev, dt, rows, "residual", residual), _ptr_of(dev, dt, gs, "gate", gate),
        _ptr_of(dev, dt, cols, "gamma_post", gamma_post), _ptr_of(dev, dt, cols, "gamma_pre", gamma_pre), _ptr_of(dev, dt, rows, "s", s),
        _ptr_of(dev, dt, rows, "xn", xn), _stream_of(stream, dev)), "moe_norm_residual")


def moe_norm_residual_backward(dims: NormDims, ds, dxn, s, y, gate, gamma_post, gamma_pre, dresidual, dy, dgate, dgamma_post, dgamma_pre, workspace,
                               stream=None):
    """Gradients of moe_norm_residual's inputs (each may be None) for the gradients ds and dxn of its results (either may be None)."""
    dt, rows, cols, gs = _sizes(dims, NormDims)
    dev = _current("y", y)
    _check(load_library().moe_norm_residual_backward(
        ctypes.byref(dims), _ptr_of(dev, dt, rows, "ds", ds), _ptr_of(dev, dt, rows, "dxn", dxn), _ptr_of(dev, dt, rows, "s", s),
        _ptr_of(dev, dt, rows, "y", y), _ptr_of(dev, dt, gs, "gate", gate), _ptr_of(dev, dt, cols, "gamma_post", gamma_post),
        _ptr_of(dev, dt, cols, "gamma_pre", gamma_pre), _ptr_of(dev, dt, rows, "dresidual", dresidual), _ptr_of(dev, dt, rows, "dy", dy),
        _ptr_of(dev, dt, gs, "dgate", dgate), _ptr_of(dev, dt, cols, "dgamma_post", dgamma_post), _ptr_of(dev, dt, cols, "dgamma_pre", dgamma_pre),
        *_workspace(dev, workspace), _stream_of(stream, dev)), "moe_norm_residual_backward")


def moe_rmsnorm(dims, x, gamma, eps: float, xn, stream=None):
    _check(load_library().moe_rmsnorm(ctypes.byref(_dims(dims)), _ptr(x), _ptr(gamma), float(eps), _ptr(xn),
                                      _stream(stream)), "moe_rmsnorm")


def moe_last_device_error(workspace, stream=None) -> int:
    """Synchronise and return (and clear) the device error status kept in the workspace."""
    return int(load_library().moe_last_device_error(_ptr(workspace), _stream(stream)))


def moe_set_trace(kernel, start_events=(), stop_events=()):
    """Record the given torch.cuda.Event pairs around every launch of ``kernel`` (a name of
    KERNELS or its id), cycling through them; empty sequences clear the trace."""
    kid = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    n = len(start_events)
    if n != len(stop_events):
        raise ValueError("start and stop event lists differ in length")
    arr = ctypes.c_void_p * max(n, 1)
    st = arr(*[e.cuda_event for e in start_events]) if n else None
    sp = arr(*[e.cuda_event for e in stop_events]) if n else None
    _check(load_library().moe_set_trace(kid, st, sp, n), "moe_set_trace")


def moe_test_set_wait(wait_ns: int = 0, suppress: int = 0):
    """Testing aid: time limit (ns, 0 = the default of ~1 s) of the bounded device waits of the
    one-token and streaming kernels, and a signal to hold back (TEST_SUPPRESS_*) so that a wait
    runs out; moe_test_set_wait() restores normal operation."""
    _check(load_library().moe_test_set_wait(int(wait_ns), int(suppress)), "moe_test_set_wait")


def moe_launch_count() -> int:
    return int(load_library().moe_launch_count())


def moe_workspace_tap(dims, tap: int) -> tuple[int, int]:
    off, nb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().moe_workspace_tap(ctypes.byref(_dims(dims)), int(tap), ctypes.byref(off), ctypes.byref(nb)),
           "moe_workspace_tap")
    return off.value, nb.value


def moe_w4_workspace_tap(dims, tap: int) -> tuple[int, int]:
    """moe_workspace_tap after moe_forward_w4 (tap 1 is fp32 for any T where K = 1)."""
    off, nb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().moe_w4_workspace_tap(ctypes.byref(_dims(dims)), int(tap), ctypes.byref(off), ctypes.byref(nb)),
           "moe_w4_workspace_tap")
    return off.value, nb.value
