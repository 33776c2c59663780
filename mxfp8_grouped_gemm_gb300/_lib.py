"""ctypes binding of libmxg.so (include/mxg.h).  Argument marshalling only:
every step of the path runs in the library's CUDA kernels.  The functions
carry the C names; torch tensors provide device memory and the stream.

There is no fallback: if the library is missing or the tensors are not CUDA
tensors, the call raises."""
from __future__ import annotations

import array
import ctypes
import itertools
import operator
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxg.so")

MXG_LAYOUT_CANONICAL = 0
MXG_LAYOUT_MMA = 1

STATUS = {
    0: "MXG_OK", 1: "MXG_ERR_ARG", 2: "MXG_ERR_SHAPE", 3: "MXG_ERR_ALIGN", 4: "MXG_ERR_ARCH",
    5: "MXG_ERR_WORKSPACE", 6: "MXG_ERR_CUDA", 16: "MXG_ERR_EXPERT_ID", 17: "MXG_ERR_OFFSETS",
    18: "MXG_ERR_TIMEOUT", 19: "MXG_ERR_INDEX",
}

EXPORTS = [
    "mxg_status_string", "mxg_device_supported", "mxg_launch_count", "mxg_route_topk",
    "mxg_route_permute_workspace_bytes", "mxg_route_permute", "mxg_mxfp8_quantize", "mxg_grouped_gemm",
    "mxg_grouped_gemm_wgrad", "mxg_mlp_saved_bytes", "mxg_mlp_workspace_bytes", "mxg_grouped_mlp_fwd",
    "mxg_grouped_mlp_bwd", "mxg_mlp_saved_view", "mxg_grouped_mlp_fwd_stage", "mxg_grouped_mlp_bwd_stage",
    "mxg_route_permute_noalloc_max_entries", "mxg_route_permute_noalloc", "mxg_mlp_group_align",
    "mxg_mlp_row_capacity", "mxg_debug_grouped_gemm_stall", "mxg_router_fwd", "mxg_router_bwd_workspace_bytes",
    "mxg_router_bwd", "mxg_mlp_bf16_saved_bytes", "mxg_mlp_bf16_workspace_bytes", "mxg_grouped_mlp_bf16_fwd",
    "mxg_grouped_mlp_bf16_bwd", "mxg_grouped_mlp_bf16_fwd_stage", "mxg_grouped_mlp_bf16_bwd_stage",
    "mxg_mlp_weight_cache_bytes", "mxg_mlp_quantize_weights", "mxg_mlp_saved_bytes_cached",
    "mxg_mlp_fp8_saved_bytes", "mxg_mlp_fp8_workspace_bytes", "mxg_grouped_mlp_fp8_fwd", "mxg_grouped_mlp_fp8_bwd",
    "mxg_grouped_mlp_fp8_fwd_stage", "mxg_grouped_mlp_fp8_bwd_stage", "mxg_mlp_fp8_saved_view",
    "mxg_mlp_workspace_view", "mxg_mlp_weight_cache_view", "mxg_bench_mxfp8_mma_peak",
    "mxg_mxfp8_grouped_rows_capacity", "mxg_mxfp8_quantize_grouped", "mxg_gather_rows", "mxg_combine",
    "mxg_mlp_grouped_saved_bytes", "mxg_mlp_grouped_workspace_bytes", "mxg_grouped_mlp_fwd_grouped",
    "mxg_router_fwd_permute", "mxg_grouped_mlp_fwd_grouped_mx",
    "mxg_balance_loss_workspace_bytes", "mxg_balance_loss_fwd", "mxg_balance_loss_bwd",
    "mxg_router_linear_bwd_workspace_bytes", "mxg_router_linear_bwd", "mxg_muon_workspace_bytes", "mxg_muon_update",
    "mxg_muon_form", "mxg_route_scores_fwd", "mxg_route_scores_bwd", "mxg_rms_norm_fwd",
    "mxg_rms_norm_bwd_workspace_bytes", "mxg_rms_norm_bwd", "mxg_grad_norm_workspace_bytes", "mxg_grad_norm",
    "mxg_grad_clip",
]

FWD_STAGES = ["permute", "quant_weights", "quant_x", "gate_up", "down", "combine"]
BWD_STAGES = ["quant_dy", "dgrad_down", "wgrad_down", "dgrad_gate_up", "wgrad_gate_up", "combine_dx", "dprobs"]


class MxgError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} -> {STATUS.get(code, code)}: {status_string(code)}")


class MlpFwdArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("x", ctypes.c_void_p), ("ids", ctypes.c_void_p),
                ("probs", ctypes.c_void_p), ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("split_sizes", ctypes.c_void_p), ("saved", ctypes.c_void_p),
                ("saved_bytes", ctypes.c_uint64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_uint64), ("save_for_backward", ctypes.c_int32),
                ("dev_status", ctypes.c_void_p), ("weight_cache", ctypes.c_void_p),
                ("weight_cache_bytes", ctypes.c_uint64)]


class MlpGroupedFwdArgs(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("split_sizes", ctypes.c_void_p), ("probs", ctypes.c_void_p),
                ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("saved", ctypes.c_void_p), ("saved_bytes", ctypes.c_uint64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_uint64), ("save_for_backward", ctypes.c_int32),
                ("dev_status", ctypes.c_void_p), ("weight_cache", ctypes.c_void_p),
                ("weight_cache_bytes", ctypes.c_uint64)]


class MlpGroupedFwdMxArgs(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("xq", ctypes.c_void_p), ("xs", ctypes.c_void_p), ("split_sizes", ctypes.c_void_p),
                ("probs", ctypes.c_void_p), ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("saved", ctypes.c_void_p), ("saved_bytes", ctypes.c_uint64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64), ("dev_status", ctypes.c_void_p),
                ("weight_cache", ctypes.c_void_p), ("weight_cache_bytes", ctypes.c_uint64)]


class MlpBwdArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("dy", ctypes.c_void_p), ("saved", ctypes.c_void_p),
                ("saved_bytes", ctypes.c_uint64), ("dx", ctypes.c_void_p), ("dw_gate_up", ctypes.c_void_p),
                ("dw_down", ctypes.c_void_p), ("dprobs", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_uint64), ("dev_status", ctypes.c_void_p),
                ("weight_cache", ctypes.c_void_p), ("weight_cache_bytes", ctypes.c_uint64),
                ("main_grad_gate_up", ctypes.c_void_p), ("main_grad_down", ctypes.c_void_p)]


class MuonArgs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("grad_f32", ctypes.c_int32), ("grad", ctypes.c_void_p), ("momentum_in", ctypes.c_void_p),
                ("momentum_out", ctypes.c_void_p), ("mu", ctypes.c_float), ("nesterov", ctypes.c_int32),
                ("steps", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("scale", ctypes.c_float), ("update", ctypes.c_void_p), ("w_in", ctypes.c_void_p),
                ("w_out", ctypes.c_void_p), ("lr", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64),
                ("dev_status", ctypes.c_void_p)]


class RmsNormFwdArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("x", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("residual_out", ctypes.c_void_p), ("residual_f32", ctypes.c_int32), ("weight_f32", ctypes.c_int32),
                ("weight", ctypes.c_void_p), ("eps", ctypes.c_float), ("layout", ctypes.c_int32),
                ("y", ctypes.c_void_p), ("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


class RmsNormBwdArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("dy", ctypes.c_void_p), ("r", ctypes.c_void_p),
                ("r_f32", ctypes.c_int32), ("weight_f32", ctypes.c_int32), ("weight", ctypes.c_void_p),
                ("rstd", ctypes.c_void_p), ("dresidual", ctypes.c_void_p), ("dx", ctypes.c_void_p),
                ("dresidual_out", ctypes.c_void_p), ("dweight", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_uint64)]


class RouteScoresFwdArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("logits", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("probs", ctypes.c_void_p)]


class RouteScoresBwdArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("logits", ctypes.c_void_p),
                ("ids", ctypes.c_void_p), ("probs", ctypes.c_void_p), ("dprobs", ctypes.c_void_p),
                ("dlogits_in", ctypes.c_void_p), ("dlogits", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class TensorRef(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("f32", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmxg.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m mxfp8_grouped_gemm_gb300.build`")
    L = ctypes.CDLL(LIB_PATH)
    I32, I64, U64, SZ, P = ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t, ctypes.c_void_p
    F32 = ctypes.c_float
    sig = {
        "mxg_status_string": (ctypes.c_char_p, [I32]),
        "mxg_device_supported": (I32, []),
        "mxg_launch_count": (U64, []),
        "mxg_route_topk": (I32, [P, I32, I32, I32, P, P, P]),
        "mxg_route_permute_workspace_bytes": (SZ, [I32, I32, I32]),
        "mxg_route_permute": (I32, [P, I32, I32, I32, P, P, P, P, P, SZ, P, P]),
        "mxg_mxfp8_quantize": (I32, [P, I32, I32, P, P, P, P, I32, P]),
        "mxg_grouped_gemm": (I32, [P, P, P, P, P, I32, I32, I32, I32, P, P, P]),
        "mxg_grouped_gemm_wgrad": (I32, [P, P, P, P, P, I32, I32, I32, I32, P, P, P]),
        "mxg_debug_grouped_gemm_stall": (I32, [P, P, P, P, P, I32, I32, I32, I32, P, U64, P, P]),
        "mxg_mlp_saved_bytes": (SZ, [I32, I32, I32, I32, I32]),
        "mxg_mlp_group_align": (I32, []),
        "mxg_mlp_row_capacity": (SZ, [I32, I32, I32]),
        "mxg_mlp_workspace_bytes": (SZ, [I32, I32, I32, I32, I32]),
        "mxg_grouped_mlp_fwd": (I32, [ctypes.POINTER(MlpFwdArgs), P]),
        "mxg_grouped_mlp_bwd": (I32, [ctypes.POINTER(MlpBwdArgs), P]),
        "mxg_mlp_saved_view": (P, [P, I32, I32, I32, I32, I32, I32]),
        "mxg_grouped_mlp_fwd_stage": (I32, [ctypes.POINTER(MlpFwdArgs), I32, P]),
        "mxg_route_permute_noalloc_max_entries": (SZ, [I32]),
        "mxg_route_permute_noalloc": (I32, [P, I32, I32, I32, P, P, P, P, P, P]),
        "mxg_grouped_mlp_bwd_stage": (I32, [ctypes.POINTER(MlpBwdArgs), I32, P]),
        "mxg_router_fwd": (I32, [P, P, I32, I32, I32, I32, P, P, P, P]),
        "mxg_mlp_bf16_saved_bytes": (SZ, [I32, I32, I32, I32, I32]),
        "mxg_mlp_bf16_workspace_bytes": (SZ, [I32, I32, I32, I32, I32]),
        "mxg_grouped_mlp_bf16_fwd": (I32, [ctypes.POINTER(MlpFwdArgs), P]),
        "mxg_grouped_mlp_bf16_bwd": (I32, [ctypes.POINTER(MlpBwdArgs), P]),
        "mxg_grouped_mlp_bf16_fwd_stage": (I32, [ctypes.POINTER(MlpFwdArgs), I32, P]),
        "mxg_grouped_mlp_bf16_bwd_stage": (I32, [ctypes.POINTER(MlpBwdArgs), I32, P]),
        "mxg_router_bwd_workspace_bytes": (SZ, [I32, I32, I32, I32]),
        "mxg_router_bwd": (I32, [P, P, P, P, P, I32, I32, I32, I32, P, P, P, SZ, P, P]),
        "mxg_mlp_weight_cache_bytes": (SZ, [I32, I32, I32]),
        "mxg_mlp_quantize_weights": (I32, [P, P, I32, I32, I32, P, SZ, P]),
        "mxg_mlp_saved_bytes_cached": (SZ, [I32, I32, I32, I32, I32]),
        "mxg_mlp_fp8_saved_bytes": (SZ, [I32, I32, I32, I32, I32]),
        "mxg_mlp_fp8_workspace_bytes": (SZ, [I32, I32, I32, I32, I32]),
        "mxg_grouped_mlp_fp8_fwd": (I32, [ctypes.POINTER(MlpFwdArgs), P]),
        "mxg_grouped_mlp_fp8_bwd": (I32, [ctypes.POINTER(MlpBwdArgs), P]),
        "mxg_grouped_mlp_fp8_fwd_stage": (I32, [ctypes.POINTER(MlpFwdArgs), I32, P]),
        "mxg_grouped_mlp_fp8_bwd_stage": (I32, [ctypes.POINTER(MlpBwdArgs), I32, P]),
        "mxg_mlp_fp8_saved_view": (P, [P, I32, I32, I32, I32, I32, I32]),
        "mxg_mlp_workspace_view": (P, [P, I32, I32, I32, I32, I32, I32]),
        "mxg_mlp_weight_cache_view": (P, [P, I32, I32, I32, I32]),
        "mxg_bench_mxfp8_mma_peak": (I32, [I32, ctypes.POINTER(ctypes.c_double), P, P]),
        "mxg_mxfp8_grouped_rows_capacity": (SZ, [I32, I32, I32]),
        "mxg_mxfp8_quantize_grouped": (I32, [P, I32, I32, P, I32, P, P, P, P, P, I32, P, P]),
        "mxg_gather_rows": (I32, [P, I64, I64, P, I32, I64, P, P, P]),
        "mxg_combine": (I32, [P, I64, P, I32, I32, I32, P, P, P]),
        "mxg_mlp_grouped_saved_bytes": (SZ, [I32, I32, I32, I32]),
        "mxg_mlp_grouped_workspace_bytes": (SZ, [I32, I32, I32, I32]),
        "mxg_grouped_mlp_fwd_grouped": (I32, [ctypes.POINTER(MlpGroupedFwdArgs), P]),
        "mxg_router_fwd_permute": (I32, [P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P, P]),
        "mxg_grouped_mlp_fwd_grouped_mx": (I32, [ctypes.POINTER(MlpGroupedFwdMxArgs), P]),
        "mxg_balance_loss_workspace_bytes": (SZ, [I32, I32]),
        "mxg_balance_loss_fwd": (I32, [P, P, P, I32, I32, I32, F32, P, P, P, P, P, SZ, P, P]),
        "mxg_balance_loss_bwd": (I32, [P, P, P, P, I32, I32, I32, F32, P, P, P, P, P, P, P]),
        "mxg_router_linear_bwd_workspace_bytes": (SZ, [I32, I32, I32]),
        "mxg_router_linear_bwd": (I32, [P, P, P, P, I32, I32, I32, P, P, P, SZ, P, P]),
        "mxg_muon_workspace_bytes": (SZ, [I32, I32, I32]),
        "mxg_muon_form": (I32, [I32, I32, I32, ctypes.POINTER(I32)]),
        "mxg_muon_update": (I32, [ctypes.POINTER(MuonArgs), P]),
        "mxg_route_scores_fwd": (I32, [P, P]),
        "mxg_route_scores_bwd": (I32, [P, P]),
        "mxg_rms_norm_fwd": (I32, [P, P]),
        "mxg_rms_norm_bwd_workspace_bytes": (SZ, [I32, I32]),
        "mxg_rms_norm_bwd": (I32, [P, P]),
        "mxg_grad_norm_workspace_bytes": (SZ, [I32]),
        "mxg_grad_norm": (I32, [P, I32, P, P, SZ, P]),
        "mxg_grad_clip": (I32, [P, I32, F32, P, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def status_string(code: int) -> str:
    return lib().mxg_status_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != 0:
        raise MxgError(fn, code)


def _ptr(t: torch.Tensor | None, dtype=None, name: str = "tensor") -> int | None:
    if t is None:
        return None
    if t.is_cuda and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        # the handle itself: building a Stream object costs more than a kernel launch
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _bits(t: torch.Tensor | None) -> torch.Tensor | None:
    return t.view(torch.int16) if t is not None and t.dtype == torch.bfloat16 else t


# ------------------------------------------------------------------ entries --

def mxg_device_supported() -> bool:
    return bool(lib().mxg_device_supported())


def mxg_launch_count() -> int:
    return int(lib().mxg_launch_count())


def mxg_route_topk(logits: torch.Tensor, k: int, ids=None, probs=None, stream=None):
    T, E = logits.shape
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device) if ids is None else ids
    probs = torch.empty((T, k), dtype=torch.float32, device=logits.device) if probs is None else probs
    _check("mxg_route_topk", lib().mxg_route_topk(_ptr(logits, torch.float32, "logits"), T, E, k,
                                                  _ptr(ids, torch.int32, "ids"), _ptr(probs, torch.float32, "probs"),
                                                  _stream(stream)))
    return ids, probs


def mxg_router_fwd(x: torch.Tensor, w_router: torch.Tensor, k: int, logits=None, ids=None, probs=None, stream=None):
    """logits = x W_r^T (fp32 out) and the top-k route on them."""
    T, H = x.shape
    E = w_router.shape[0]
    dev = x.device
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if logits is None else logits
    ids = torch.empty((T, k), dtype=torch.int32, device=dev) if ids is None else ids
    probs = torch.empty((T, k), dtype=torch.float32, device=dev) if probs is None else probs
    _check("mxg_router_fwd", lib().mxg_router_fwd(_ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.bfloat16, "w_router"),
                                                  T, H, E, k, _ptr(logits, torch.float32, "logits"),
                                                  _ptr(ids, torch.int32, "ids"), _ptr(probs, torch.float32, "probs"),
                                                  _stream(stream)))
    return logits, ids, probs


def mxg_router_bwd_workspace_bytes(T, H, E, k) -> int:
    return int(lib().mxg_router_bwd_workspace_bytes(T, H, E, k))


def mxg_router_bwd(x, w_router, ids, probs, dprobs, dx, dev_status, dw_router=None, workspace=None, stream=None):
    """Adds the router's term to dx (in place) and returns dW_r (fp32)."""
    T, H = x.shape
    E = w_router.shape[0]
    k = ids.shape[1]
    dev = x.device
    dw_router = torch.empty((E, H), dtype=torch.float32, device=dev) if dw_router is None else dw_router
    nbytes = mxg_router_bwd_workspace_bytes(T, H, E, k)
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if workspace is None else workspace
    _check("mxg_router_bwd", lib().mxg_router_bwd(
        _ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.bfloat16, "w_router"), _ptr(ids, torch.int32, "ids"),
        _ptr(probs, torch.float32, "probs"), _ptr(dprobs, torch.float32, "dprobs"), T, H, E, k,
        _ptr(dx, torch.bfloat16, "dx"), _ptr(dw_router, torch.float32, "dw_router"), _ptr(workspace), workspace.numel(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return dw_router


def _empty(shape, dtype, device, stream):
    """Memory for a call on `stream`: from that stream's own pool, so that neither what used the memory before
    nor what uses it next overlaps the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=device)


class _ScratchCache(threading.local):
    """Small scratch kept per thread, device and stream: making and dropping a tensor takes longer than a launch.
    Calls of one thread on one stream follow one another, so they can share it.  A stream is known by its handle, as
    in torch's allocator: one that is not torch's is destroyed only after its work has ended."""
    BYTES = 1 << 20
    MOST = 64                              # as many streams; the oldest makes room (its memory goes to its stream's pool)

    def __init__(self):
        self.kept = {}

    def get(self, device, handle):
        key = (device.index, handle)
        t = self.kept.get(key)
        if t is None:
            if len(self.kept) >= self.MOST:
                del self.kept[next(iter(self.kept))]
            t = self.kept[key] = torch.empty(self.BYTES, dtype=torch.uint8, device=device)
        return t


_scratch_cache = _ScratchCache()


def _call_with_scratch(name: str, call, bytes_of, workspace, device, stream):
    """call(pointer, bytes, stream handle) -> status, with the caller's workspace, the kept scratch, or, where that is
    too small, the stream is not the current one or a graph is being captured, memory of its own."""
    handle = _stream(stream)
    if workspace is None and stream is None and not torch.cuda.is_current_stream_capturing():
        t = _scratch_cache.get(device, handle)
        status = call(t.data_ptr(), _ScratchCache.BYTES, handle)
        if status != 5:                                # MXG_ERR_WORKSPACE: nothing was launched
            return _check(name, status)
    if workspace is None:
        workspace = _empty(max(bytes_of(), 32), torch.uint8, device, stream)
    _check(name, call(_ptr(workspace, None, "workspace"), workspace.numel(), handle))


def _shape(t: torch.Tensor | None, shape: tuple, name: str):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _mask_ptr(mask: torch.Tensor | None, T: int) -> int | None:
    if mask is None:
        return None
    if mask.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"token_mask must be bool or uint8, got {mask.dtype}")
    _shape(mask, (T,), "token_mask")
    return _ptr(mask, None, "token_mask")


def mxg_balance_loss_workspace_bytes(T, E) -> int:
    return int(lib().mxg_balance_loss_workspace_bytes(T, E))


def mxg_balance_loss_fwd(logits, ids, coef: float, dev_status, token_mask=None, loss=None, counts=None, prob_sums=None,
                         n_tokens=None, workspace=None, stream=None):
    """Balance loss of the router -> (loss fp32 [1], counts int32 [E], prob_sums fp32 [E], n_tokens int32 [1])."""
    T, E = logits.shape
    k = ids.shape[-1]
    dev = logits.device
    _shape(ids, (T, k), "ids")
    loss = _empty(1, torch.float32, dev, stream) if loss is None else loss
    counts = _empty(E, torch.int32, dev, stream) if counts is None else counts
    prob_sums = _empty(E, torch.float32, dev, stream) if prob_sums is None else prob_sums
    n_tokens = _empty(1, torch.int32, dev, stream) if n_tokens is None else n_tokens
    _shape(loss, (1,), "loss")
    _shape(counts, (E,), "counts")
    _shape(prob_sums, (E,), "prob_sums")
    _shape(n_tokens, (1,), "n_tokens")
    args = (_ptr(logits, torch.float32, "logits"), _ptr(ids, torch.int32, "ids"), _mask_ptr(token_mask, T), T, E, k, coef,
            _ptr(loss, torch.float32, "loss"), _ptr(counts, torch.int32, "counts"),
            _ptr(prob_sums, torch.float32, "prob_sums"), _ptr(n_tokens, torch.int32, "n_tokens"))
    status = _ptr(dev_status, torch.int32, "dev_status")
    _call_with_scratch("mxg_balance_loss_fwd",
                       lambda ws, n, s: lib().mxg_balance_loss_fwd(*args, ws, n, status, s),
                       lambda: mxg_balance_loss_workspace_bytes(T, E), workspace, dev, stream)
    return loss, counts, prob_sums, n_tokens


def mxg_balance_loss_bwd(logits, counts, n_tokens, k: int, coef: float, dev_status, dloss=None, token_mask=None,
                         route=None, dlogits=None, stream=None):
    """Gradient of the balance loss on the logits, fp32 [T, E]; route = (ids, probs, dprobs) adds the route's own."""
    T, E = logits.shape
    dlogits = _empty((T, E), torch.float32, logits.device, stream) if dlogits is None else dlogits
    ids, probs, dprobs = (None, None, None) if route is None else route
    _shape(dlogits, (T, E), "dlogits")
    _shape(counts, (E,), "counts")
    _shape(n_tokens, (1,), "n_tokens")
    _shape(dloss, (1,), "dloss")
    _shape(ids, (T, k), "ids")
    _shape(probs, (T, k), "probs")
    _shape(dprobs, (T, k), "dprobs")
    _check("mxg_balance_loss_bwd", lib().mxg_balance_loss_bwd(
        _ptr(logits, torch.float32, "logits"), _mask_ptr(token_mask, T), _ptr(counts, torch.int32, "counts"),
        _ptr(n_tokens, torch.int32, "n_tokens"), T, E, k, coef, _ptr(dloss, torch.float32, "dloss"),
        _ptr(ids, torch.int32, "ids"), _ptr(probs, torch.float32, "probs"), _ptr(dprobs, torch.float32, "dprobs"),
        _ptr(dlogits, torch.float32, "dlogits"), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return dlogits


def mxg_router_linear_bwd_workspace_bytes(T, H, E) -> int:
    return int(lib().mxg_router_linear_bwd_workspace_bytes(T, H, E))


def mxg_router_linear_bwd(x, w_router, dlogits, dx_in, dev_status, dx=None, dw_router=None, workspace=None,
                          stream=None):
    """Router linear layer's backward for dense logit gradients: (dx = dx_in + dlogits W_r, dW_r = dlogits^T x).
    dx_in None: no other gradient; dx may be dx_in."""
    T, H = x.shape
    E = w_router.shape[0]
    dev = x.device
    dx = _empty((T, H), torch.bfloat16, dev, stream) if dx is None else dx
    dw_router = _empty((E, H), torch.float32, dev, stream) if dw_router is None else dw_router
    _shape(w_router, (E, H), "w_router")
    _shape(dlogits, (T, E), "dlogits")
    _shape(dx_in, (T, H), "dx_in")
    _shape(dx, (T, H), "dx")
    _shape(dw_router, (E, H), "dw_router")
    args = (_ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.bfloat16, "w_router"),
            _ptr(dlogits, torch.float32, "dlogits"), _ptr(dx_in, torch.bfloat16, "dx_in"), T, H, E,
            _ptr(dx, torch.bfloat16, "dx"), _ptr(dw_router, torch.float32, "dw_router"))
    status = _ptr(dev_status, torch.int32, "dev_status")
    _call_with_scratch("mxg_router_linear_bwd",
                       lambda ws, n, s: lib().mxg_router_linear_bwd(*args, ws, n, status, s),
                       lambda: mxg_router_linear_bwd_workspace_bytes(T, H, E), workspace, dev, stream)
    return dx, dw_router


def mxg_muon_workspace_bytes(batch, rows, cols) -> int:
    return int(lib().mxg_muon_workspace_bytes(batch, rows, cols))


def mxg_muon_form(batch, rows, cols) -> dict:
    """The form that an update of these sizes takes on the current device: `cluster` CTAs keep a matrix on the chip, or,
    where that is 0, products in tiles of `tile` columns, `shares` CTAs to a tile of X X^T; X in `parts` fp16 numbers."""
    form = (ctypes.c_int * 4)()
    _check("mxg_muon_form", lib().mxg_muon_form(batch, rows, cols, form))
    return dict(zip(("cluster", "tile", "shares", "parts"), form))


MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def mxg_muon_update(grad, dev_status, momentum=None, momentum_out=None, mu: float = 0.95, nesterov: bool = True,
                    steps: int = 5, coefficients=MUON_COEFFICIENTS, scale: float = 1.0, update=None, weights=None,
                    weights_out=None, lr: float = 0.0, weight_decay: float = 0.0, workspace=None, stream=None):
    """Orthogonalised momentum update of grad [batch, rows, cols] (or [rows, cols]; bf16 or fp32).

    momentum (fp32) is read and momentum_out written (momentum itself if not given); with momentum_out alone the
    momentum starts at zero, with neither there is none.  weights (bf16): the new weights go to weights_out
    (weights itself if not given) and are returned; otherwise the bf16 update is (also where `update` is given)."""
    shape = tuple(grad.shape)
    if grad.dim() not in (2, 3):
        raise ValueError(f"grad must be [rows, cols] or [batch, rows, cols], got {list(shape)}")
    if grad.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"grad must be bfloat16 or float32, got {grad.dtype}")
    if weights_out is not None and weights is None:
        raise ValueError("weights_out needs weights")
    batch, rows, cols = shape if grad.dim() == 3 else (1, *shape)
    dev = grad.device
    momentum_out = momentum if momentum_out is None else momentum_out
    weights_out = weights if weights_out is None else weights_out
    if update is None and weights is None:
        update = _empty(shape, torch.bfloat16, dev, stream)
    for name, t in (("momentum", momentum), ("momentum_out", momentum_out), ("update", update), ("weights", weights),
                    ("weights_out", weights_out)):
        _shape(t, shape, name)
    a, b, c = coefficients
    args = MuonArgs(batch=batch, rows=rows, cols=cols, grad_f32=int(grad.dtype == torch.float32),
                    grad=_ptr(grad, None, "grad"), momentum_in=_ptr(momentum, torch.float32, "momentum"),
                    momentum_out=_ptr(momentum_out, torch.float32, "momentum_out"), mu=mu, nesterov=int(nesterov),
                    steps=steps, a=a, b=b, c=c, scale=scale, update=_ptr(update, torch.bfloat16, "update"),
                    w_in=_ptr(weights, torch.bfloat16, "weights"),
                    w_out=_ptr(weights_out, torch.bfloat16, "weights_out"), lr=lr, weight_decay=weight_decay,
                    dev_status=_ptr(dev_status, torch.int32, "dev_status"))

    def call(ws, n, s):
        args.workspace, args.workspace_bytes = ws, n
        return lib().mxg_muon_update(ctypes.byref(args), s)

    _call_with_scratch("mxg_muon_update", call, lambda: mxg_muon_workspace_bytes(batch, rows, cols), workspace, dev,
                       stream)
    return update if weights is None else weights_out


MXG_SCORE = {"softmax": 0, "sigmoid": 1}


def _score(name) -> int:
    if name not in MXG_SCORE:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {name!r}")
    return MXG_SCORE[name]


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {list(t.shape)}")
    return t.shape


def _real(t: torch.Tensor | None, name: str):
    if t is not None and t.dtype is not torch.bfloat16 and t.dtype is not torch.float32:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _pointers(names, tensors, dtypes, shapes) -> list:
    """Addresses of tensors (0 for None) that have these types and shapes (None: any) and are contiguous and on the
    current device, where the library runs.  Small calls take as long as this, so it looks at each tensor once."""
    out, dev = [], None
    add = out.append
    for t, dtype, shape in zip(tensors, dtypes, shapes):
        if t is None:
            add(0)
            continue
        d = t.get_device()
        if dev is None and d >= 0:
            dev = torch._C._cuda_getDevice()
        if d != dev or t.dtype is not dtype or (shape is not None and t.shape != shape) or not t.is_contiguous():
            _refuse(names, tensors, dtypes, shapes)
        add(t.data_ptr())
    return out


def _refuse(names, tensors, dtypes, shapes):
    for name, t, shape in zip(names, tensors, shapes):
        if shape is not None:
            _shape(t, shape, name)
    for name, t, dtype in zip(names, tensors, dtypes):
        _ptr(t, dtype, name)
    here = torch._C._cuda_getDevice()
    for name, t in zip(names, tensors):
        if t is not None and t.get_device() != here:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{here}")


# the C structures as the bytes that a call passes: one call of struct where ctypes takes a step per field
_PACK_ROUTE_FWD = struct.Struct("@iiiiiiiifPPPP")
_PACK_ROUTE_BWD = struct.Struct("@iiiiifPPPPPPP")
_ROUTE_FWD = ("logits", "bias", "ids", "probs")
_ROUTE_FWD_TYPES = (torch.float32, torch.float32, torch.int32, torch.float32)


def mxg_route_scores_fwd(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
                         group_top: int = 2, renormalize: bool = True, scale: float = 1.0, ids=None, probs=None,
                         stream=None):
    """Routing by softmax or sigmoid scores of logits [T, E] -> (ids int32 [T, k], probs fp32 [T, k]).

    bias (fp32 [E]) is added for the choice alone; of `groups` groups of experts the `top_groups` with the largest sums
    of their group_top largest scores take part; the weights are the chosen scores, renormalised or not, times scale."""
    T, E = _matrix(logits, "logits")
    kind = _score(score)
    ids = _empty((T, k), torch.int32, logits.device, stream) if ids is None else ids
    probs = _empty((T, k), torch.float32, logits.device, stream) if probs is None else probs
    z, b, i, p = _pointers(_ROUTE_FWD, (logits, bias, ids, probs), _ROUTE_FWD_TYPES, (None, (E,), (T, k), (T, k)))
    args = _PACK_ROUTE_FWD.pack(T, E, k, kind, groups, top_groups, group_top, renormalize, scale, z, b, i, p)
    _check("mxg_route_scores_fwd", lib().mxg_route_scores_fwd(args, _stream(stream)))
    return ids, probs


_ROUTE_BWD = ("logits", "ids", "probs", "dprobs", "dlogits_in", "dlogits", "dev_status")
_ROUTE_BWD_TYPES = (torch.float32, torch.int32, torch.float32, torch.float32, torch.float32, torch.float32, torch.int32)


def mxg_route_scores_bwd(logits, ids, probs, dprobs, dev_status, score: str = "softmax", renormalize: bool = True,
                         scale: float = 1.0, dlogits_in=None, dlogits=None, stream=None):
    """Gradient of mxg_route_scores_fwd's weights on the logits, dense fp32 [T, E], added to dlogits_in if given (which
    may be dlogits)."""
    T, E = _matrix(logits, "logits")
    k = _matrix(ids, "ids")[1]
    kind = _score(score)
    dlogits = _empty((T, E), torch.float32, logits.device, stream) if dlogits is None else dlogits
    z, i, p, dp, add, d, st = _pointers(_ROUTE_BWD, (logits, ids, probs, dprobs, dlogits_in, dlogits, dev_status),
                                        _ROUTE_BWD_TYPES, (None, (T, k), (T, k), (T, k), (T, E), (T, E), None))
    args = _PACK_ROUTE_BWD.pack(T, E, k, kind, renormalize, scale, z, i, p, dp, add, d, st)
    _check("mxg_route_scores_bwd", lib().mxg_route_scores_bwd(args, _stream(stream)))
    return dlogits


_PACK_NORM_FWD = struct.Struct("@iiPPPiiPfiPPPP")
_PACK_NORM_BWD = struct.Struct("@iiPPiiPPPPPPPQ")
_NORM_FWD = ("x", "weight", "residual", "residual_out", "y", "q", "s", "rstd")


def mxg_rms_norm_fwd(x, weight, eps: float = 1e-6, residual=None, residual_out=None, y=None, q=None, s=None, rstd=None,
                     codes: bool = False, bf16: bool = True, layout: int = MXG_LAYOUT_CANONICAL, stream=None) -> dict:
    """Residual addition and root-mean-square norm of x bf16 [T, H] -> {'y', 'rstd'}, with a residual 'residual' (the
    sum, residual_out), with codes (or q and s given) 'q' uint8 [T, H] and 's' uint8 (T * H / 32 bytes, `layout`).

    residual and weight are bf16 or fp32.  residual_out may be residual, y may be x.  bf16 False: codes alone, no y."""
    T, H = TH = _matrix(x, "x")
    dev = x.device
    if (q is None) != (s is None):
        raise ValueError("q and s are given together")
    if residual_out is not None and residual is None:
        raise ValueError("residual_out needs residual")
    if not bf16 and y is not None:
        raise ValueError("y is given but bf16 is False")
    _real(residual, "residual")
    _real(weight, "weight")
    stream_type = torch.float32 if residual is None else residual.dtype
    y = _empty(TH, torch.bfloat16, dev, stream) if y is None and bf16 else y
    rstd = _empty(T, torch.float32, dev, stream) if rstd is None else rstd
    if residual is not None and residual_out is None:
        residual_out = _empty(TH, stream_type, dev, stream)
    if codes and q is None:
        q = _empty(TH, torch.uint8, dev, stream)
        s = _empty((T, H // 32), torch.uint8, dev, stream)
    if s is not None and s.numel() != T * H // 32:
        raise ValueError(f"s must have {T * H // 32} elements, got {s.numel()}")
    px, pw, pr, po, py, pq, ps, pn = _pointers(
        _NORM_FWD, (x, weight, residual, residual_out, y, q, s, rstd),
        (torch.bfloat16, weight.dtype, stream_type, stream_type, torch.bfloat16, torch.uint8, torch.uint8, torch.float32),
        (None, (H,), TH, TH, TH, TH, None, (T,)))
    args = _PACK_NORM_FWD.pack(T, H, px, pr, po, residual is not None and stream_type is torch.float32,
                               weight.dtype is torch.float32, pw, eps, layout, py, pq, ps, pn)
    _check("mxg_rms_norm_fwd", lib().mxg_rms_norm_fwd(args, _stream(stream)))
    out = {"rstd": rstd}
    if y is not None:
        out["y"] = y
    if residual is not None:
        out["residual"] = residual_out
    if q is not None:
        out["q"], out["s"] = q, s
    return out


def mxg_rms_norm_bwd_workspace_bytes(T, H) -> int:
    return int(lib().mxg_rms_norm_bwd_workspace_bytes(T, H))


_NORM_BWD = ("dy", "r", "weight", "rstd", "dresidual", "dx", "dresidual_out", "dweight")


def mxg_rms_norm_bwd(dy, r, weight, rstd, dresidual=None, dx=None, dresidual_out=None, dweight=None, workspace=None,
                     stream=None):
    """Backward of mxg_rms_norm_fwd for r = its 'residual' (or x, without one), bf16 or fp32 -> (dx bf16 [T, H],
    dresidual_out fp32 [T, H] where r is fp32, else None, dweight fp32 [H]).

    dresidual (r's type) is the gradient that reaches the sum from elsewhere.  With a bf16 residual, dx is the gradient
    of x and of the residual alike.  dx may be dy or dresidual, dresidual_out may be dresidual."""
    T, H = TH = _matrix(dy, "dy")
    dev = dy.device
    _real(r, "r")
    _real(weight, "weight")
    f32 = r.dtype is torch.float32
    if dresidual_out is not None and not f32:
        raise ValueError("dresidual_out is for an fp32 residual: dx is the gradient of a bf16 one")
    dx = _empty(TH, torch.bfloat16, dev, stream) if dx is None else dx
    if f32 and dresidual_out is None:
        dresidual_out = _empty(TH, torch.float32, dev, stream)
    dweight = _empty(H, torch.float32, dev, stream) if dweight is None else dweight
    py, pr, pw, pn, pd, px, po, pg = _pointers(
        _NORM_BWD, (dy, r, weight, rstd, dresidual, dx, dresidual_out, dweight),
        (torch.bfloat16, r.dtype, weight.dtype, torch.float32, r.dtype, torch.bfloat16, torch.float32, torch.float32),
        (None, TH, (H,), (T,), TH, TH, TH, (H,)))
    w32 = weight.dtype is torch.float32

    def call(ws, n, st):
        return lib().mxg_rms_norm_bwd(_PACK_NORM_BWD.pack(T, H, py, pr, f32, w32, pw, pn, pd, px, po, pg, ws, n), st)

    _call_with_scratch("mxg_rms_norm_bwd", call, lambda: mxg_rms_norm_bwd_workspace_bytes(T, H), workspace, dev, stream)
    return dx, dresidual_out, dweight


def mxg_grad_norm_workspace_bytes(n) -> int:
    return int(lib().mxg_grad_norm_workspace_bytes(n))


_data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel
_get_device, _is_contiguous, _dtype = torch.Tensor.get_device, torch.Tensor.is_contiguous, operator.attrgetter("dtype")
_REAL = {torch.float32, torch.bfloat16}


def _tensor_refs(grads, out):
    """The library's table of the tensors (mxg_tensor, four 64-bit words each); out None: no outputs.  A model's worth of
    small gradients takes longer here than on the GPU, so the tensors are asked for one thing after the other, without a
    loop over them."""
    n = len(grads)
    if n == 0:
        raise ValueError("no gradients given")
    if out is not None and len(out) != n:
        raise ValueError(f"{n} gradients but {len(out)} outputs")
    types, sizes, ptrs = list(map(_dtype, grads)), list(map(_numel, grads)), list(map(_data_ptr, grads))
    devices = set(map(_get_device, grads))
    if devices != {torch._C._cuda_getDevice() if grads[0].is_cuda else None} or not _REAL.issuperset(types) or not all(
            map(_is_contiguous, grads)):
        for i, t in enumerate(grads):
            _real(t, f"grads[{i}]")
            _refuse((f"grads[{i}]",), (t,), (t.dtype,), (None,))
    to = ptrs
    if out is not None and out is not grads:
        if (set(map(_get_device, out)) != devices or list(map(_dtype, out)) != types or list(map(_numel, out)) != sizes
                or not all(map(_is_contiguous, out))):
            for i, (t, o, size) in enumerate(zip(grads, out, sizes)):
                if o.numel() != size:
                    raise ValueError(f"out[{i}] must have {size} elements, got {list(o.shape)}")
                _refuse((f"out[{i}]",), (o,), (t.dtype,), (None,))
        to = list(map(_data_ptr, out))
    if out is not None and len({*ptrs, *to}) != (n if to is ptrs else 2 * n):     # an address that stands twice
        used = [p for p, size in zip(to, sizes) if size]                          # (without elements it may)
        if len(set(used)) != len(used):
            raise ValueError("a tensor is listed twice as an output")
        # an output in the place of another gradient, which the pass still reads
        at = {p: i for i, (p, size) in enumerate(zip(ptrs, sizes)) if size}
        for i, (p, size) in enumerate(zip(to, sizes)):
            if size and at.get(p, i) != i:
                raise ValueError(f"out[{i}] is another gradient (grads[{at[p]}])")
    f32 = torch.float32
    words = itertools.chain.from_iterable(zip(ptrs, to, sizes, [d is f32 for d in types]))
    return array.array("q", words), n


def _norm_ptr(norm, name: str) -> int:
    return _pointers((name,), (norm,), (torch.float32,), ((1,),))[0]


def mxg_grad_norm(grads, norm=None, workspace=None, stream=None):
    """Norm over all tensors of a list (bf16, fp32; contiguous, any shapes) -> fp32 [1]."""
    refs, n = _tensor_refs(grads, None)
    dev = grads[0].device
    if norm is None:
        norm = _empty(1, torch.float32, dev, stream)
        to = norm.data_ptr()
    else:
        to = _norm_ptr(norm, "norm")
    table = refs.buffer_info()[0]
    _call_with_scratch("mxg_grad_norm", lambda ws, b, st: lib().mxg_grad_norm(table, n, to, ws, b, st),
                       lambda: mxg_grad_norm_workspace_bytes(n), workspace, dev, stream)
    return norm


def mxg_grad_clip(grads, max_norm: float, out=None, norm=None, norm_out=None, workspace=None, stream=None):
    """Gradients times min(1, max_norm / norm) -> (norm fp32 [1], outputs), into `out` (a list like grads) or, without
    one, in place.  norm: fp32 [1] to clip by, e.g. joined over ranks; else the norm over grads is taken (norm_out).
    An output has its gradient's type and number of elements, in the order of the memory (a flat view will do); it may be
    that gradient and overlaps no other tensor."""
    if norm is not None and norm_out is not None:
        raise ValueError("norm_out is for the norm that is taken here")
    out = grads if out is None else out
    refs, n = _tensor_refs(grads, out)
    table = refs.buffer_info()[0]
    if norm is not None:
        by = _norm_ptr(norm, "norm")
        _check("mxg_grad_clip", lib().mxg_grad_clip(table, n, max_norm, by, None, None, 0, _stream(stream)))
        return norm, out
    dev = grads[0].device
    if norm_out is None:
        norm_out = _empty(1, torch.float32, dev, stream)
        to = norm_out.data_ptr()
    else:
        to = _norm_ptr(norm_out, "norm_out")
    _call_with_scratch("mxg_grad_clip", lambda ws, b, st: lib().mxg_grad_clip(table, n, max_norm, None, to, ws, b, st),
                       lambda: mxg_grad_norm_workspace_bytes(n), workspace, dev, stream)
    return norm_out, out


def mxg_route_permute(ids: torch.Tensor, E: int, dev_status: torch.Tensor, stream=None) -> dict:
    T, k = ids.shape
    dev = ids.device
    ws_bytes = int(lib().mxg_route_permute_workspace_bytes(T, k, E))
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    out = {"split_sizes": torch.empty(E, dtype=torch.int32, device=dev),
           "src_of_row": torch.empty(T * k, dtype=torch.int32, device=dev),
           "row_of_src": torch.empty(T * k, dtype=torch.int32, device=dev),
           "padded_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev)}
    _check("mxg_route_permute", lib().mxg_route_permute(
        _ptr(ids, torch.int32, "ids"), T, k, E, _ptr(out["split_sizes"]), _ptr(out["src_of_row"]),
        _ptr(out["row_of_src"]), _ptr(out["padded_offsets"]), _ptr(ws), ws_bytes,
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return out


def mxfp8_scale_bytes(rows: int, cols: int) -> int:
    return rows * cols // 32


def mxg_mxfp8_quantize(x: torch.Tensor, row: bool = True, col: bool = False, layout: int = MXG_LAYOUT_CANONICAL,
                       stream=None) -> dict:
    """x bf16 [rows, cols] -> {'q_row','s_row'} and/or {'q_col','s_col'} (uint8)."""
    rows, cols = x.shape
    dev = x.device
    out = {}
    if row:
        out["q_row"] = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        out["s_row"] = torch.empty(rows * cols // 32, dtype=torch.uint8, device=dev)
    if col:
        out["q_col"] = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
        out["s_col"] = torch.empty(rows * cols // 32, dtype=torch.uint8, device=dev)
    _check("mxg_mxfp8_quantize", lib().mxg_mxfp8_quantize(
        _ptr(_bits(x), None, "x"), rows, cols, _ptr(out.get("q_row")), _ptr(out.get("s_row")),
        _ptr(out.get("q_col")), _ptr(out.get("s_col")), layout, _stream(stream)))
    return out


def mxg_grouped_gemm(a, sa, b, sb, padded_offsets, E: int, N: int, K: int, dev_status, d=None, stream=None):
    m_cap = a.shape[0]
    d = torch.empty((m_cap, N), dtype=torch.bfloat16, device=a.device) if d is None else d
    _check("mxg_grouped_gemm", lib().mxg_grouped_gemm(
        _ptr(a, torch.uint8, "a"), _ptr(sa, torch.uint8, "sa"), _ptr(b, torch.uint8, "b"), _ptr(sb, torch.uint8, "sb"),
        _ptr(padded_offsets, torch.int32, "padded_offsets"), E, m_cap, N, K, _ptr(_bits(d)),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return d


def mxg_grouped_gemm_wgrad(a, sa, b, sb, padded_offsets, E: int, dev_status, d=None, stream=None):
    M, t_cap = a.shape
    N = b.shape[0]
    d = torch.empty((E, M, N), dtype=torch.bfloat16, device=a.device) if d is None else d
    _check("mxg_grouped_gemm_wgrad", lib().mxg_grouped_gemm_wgrad(
        _ptr(a, torch.uint8, "a"), _ptr(sa, torch.uint8, "sa"), _ptr(b, torch.uint8, "b"), _ptr(sb, torch.uint8, "sb"),
        _ptr(padded_offsets, torch.int32, "padded_offsets"), E, M, N, t_cap, _ptr(_bits(d)),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return d


def mxg_mlp_group_align() -> int:
    return int(lib().mxg_mlp_group_align())


def mxg_mlp_row_capacity(T, k, E) -> int:
    return int(lib().mxg_mlp_row_capacity(T, k, E))


def mxg_mlp_saved_bytes(T, H, I, E, k) -> int:
    return int(lib().mxg_mlp_saved_bytes(T, H, I, E, k))


def mxg_mlp_workspace_bytes(T, H, I, E, k) -> int:
    return int(lib().mxg_mlp_workspace_bytes(T, H, I, E, k))


def mxg_mlp_bf16_saved_bytes(T, H, I, E, k) -> int:
    return int(lib().mxg_mlp_bf16_saved_bytes(T, H, I, E, k))


def mxg_mlp_bf16_workspace_bytes(T, H, I, E, k) -> int:
    return int(lib().mxg_mlp_bf16_workspace_bytes(T, H, I, E, k))


def mxg_mlp_fp8_saved_bytes(T, H, I, E, k) -> int:
    return int(lib().mxg_mlp_fp8_saved_bytes(T, H, I, E, k))


def mxg_mlp_fp8_workspace_bytes(T, H, I, E, k) -> int:
    return int(lib().mxg_mlp_fp8_workspace_bytes(T, H, I, E, k))


def mxg_mlp_saved_view(saved: torch.Tensor, T, H, I, E, k, which: int) -> int:
    return int(lib().mxg_mlp_saved_view(_ptr(saved), T, H, I, E, k, which) or 0)


def mxg_mlp_workspace_view(workspace: torch.Tensor, T, H, I, E, k, which: int) -> int:
    return int(lib().mxg_mlp_workspace_view(_ptr(workspace), T, H, I, E, k, which) or 0)


class WeightCache:
    """The MXFP8 weights of one expert MLP (all four orientations), written by
    mxg_mlp_quantize_weights and read by forward / backward calls until the
    weights change."""

    def __init__(self, H: int, I: int, E: int, device="cuda"):
        n = int(lib().mxg_mlp_weight_cache_bytes(H, I, E))
        if n == 0:
            raise ValueError(f"unsupported weight shape H={H} I={I} E={E}")
        self.H, self.I, self.E = H, I, E
        self.buffer = torch.empty(n, dtype=torch.uint8, device=device)


def mxg_mlp_saved_bytes_cached(T, H, I, E, k) -> int:
    return int(lib().mxg_mlp_saved_bytes_cached(T, H, I, E, k))


def mxg_mlp_quantize_weights(w_gate_up, w_down, cache: WeightCache | None = None, stream=None) -> WeightCache:
    """Quantise the bf16 expert weights into a weight cache (allocated if not given)."""
    E, N2, H = w_gate_up.shape
    I = N2 // 2
    if tuple(w_down.shape) != (E, H, I):
        raise ValueError(f"w_down must be [E, H, I] = {(E, H, I)}, got {tuple(w_down.shape)}")
    cache = WeightCache(H, I, E, w_gate_up.device) if cache is None else cache
    if (cache.H, cache.I, cache.E) != (H, I, E):
        raise ValueError("weight cache was made for another shape")
    _check("mxg_mlp_quantize_weights",
           lib().mxg_mlp_quantize_weights(_ptr(_bits(w_gate_up), torch.int16, "w_gate_up"),
                                          _ptr(_bits(w_down), torch.int16, "w_down"), H, I, E,
                                          _ptr(cache.buffer, torch.uint8, "cache"), cache.buffer.numel(),
                                          _stream(stream)))
    return cache


def mxg_grouped_mlp_fwd(x, ids, probs, w_gate_up, w_down, saved, workspace, dev_status, y=None, split_sizes=None,
                        save_for_backward: bool = True, stream=None, stage: int | None = None, bf16: bool = False,
                        weight_cache: WeightCache | None = None, fp8: bool = False):
    """Full forward, or one stage of it (FWD_STAGES index) when ``stage`` is given
    (``bf16``: the BF16 path, mxg_grouped_mlp_bf16_fwd).  With ``weight_cache``
    the weights are read from it and w_gate_up / w_down may be None."""
    T, H = x.shape
    k = ids.shape[1]
    if weight_cache is not None:
        E, I = weight_cache.E, weight_cache.I
    else:
        E, N2, _ = w_gate_up.shape
        I = N2 // 2
    y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device) if y is None else y
    split_sizes = torch.empty(E, dtype=torch.int32, device=x.device) if split_sizes is None else split_sizes
    a = MlpFwdArgs(T, H, I, E, k, _ptr(_bits(x), torch.int16, "x"), _ptr(ids, torch.int32, "ids"),
                   _ptr(probs, torch.float32, "probs"), _ptr(_bits(w_gate_up), torch.int16, "w_gate_up"),
                   _ptr(_bits(w_down), torch.int16, "w_down"), _ptr(_bits(y)), _ptr(split_sizes, torch.int32),
                   _ptr(saved, torch.uint8, "saved"), saved.numel(), _ptr(workspace, torch.uint8, "workspace"),
                   workspace.numel(), 1 if save_for_backward else 0, _ptr(dev_status, torch.int32, "dev_status"),
                   None if weight_cache is None else _ptr(weight_cache.buffer, torch.uint8, "weight_cache"),
                   0 if weight_cache is None else weight_cache.buffer.numel())
    name = "mxg_grouped_mlp_bf16_fwd" if bf16 else ("mxg_grouped_mlp_fp8_fwd" if fp8 else "mxg_grouped_mlp_fwd")
    if stage is None:
        _check(name, getattr(lib(), name)(ctypes.byref(a), _stream(stream)))
    else:
        _check(name + "_stage", getattr(lib(), name + "_stage")(ctypes.byref(a), stage, _stream(stream)))
    return y, split_sizes


def mxg_grouped_mlp_bwd(dy, saved, workspace, dev_status, E: int, I: int, k: int, dx=None, dw_gate_up=None,
                        dw_down=None, dprobs=None, stream=None, stage: int | None = None, bf16: bool = False,
                        weight_cache: WeightCache | None = None, main_grad=None, fp8: bool = False):
    """Full backward, or one stage of it (BWD_STAGES index) when ``stage`` is given
    (``bf16``: the BF16 path, mxg_grouped_mlp_bf16_bwd).  ``weight_cache``: the
    cache the forward used.  ``main_grad`` = (fp32 [E, 2I, H], fp32 [E, H, I]):
    the weight gradients are added into these and returned in place of dW."""
    T, H = dy.shape
    dev = dy.device
    dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if dx is None else dx
    if main_grad is not None:
        mg_gu, mg_d = main_grad
        if tuple(mg_gu.shape) != (E, 2 * I, H) or tuple(mg_d.shape) != (E, H, I):
            raise ValueError("main_grad must be fp32 [E, 2I, H] and [E, H, I]")
        dw_gate_up = dw_down = None
    else:
        mg_gu = mg_d = None
        dw_gate_up = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=dev) if dw_gate_up is None else dw_gate_up
        dw_down = torch.empty((E, H, I), dtype=torch.bfloat16, device=dev) if dw_down is None else dw_down
    dprobs = torch.empty((T, k), dtype=torch.float32, device=dev) if dprobs is None else dprobs
    a = MlpBwdArgs(T, H, I, E, k, _ptr(_bits(dy), torch.int16, "dy"), _ptr(saved, torch.uint8, "saved"),
                   saved.numel(), _ptr(_bits(dx)), _ptr(_bits(dw_gate_up)), _ptr(_bits(dw_down)),
                   _ptr(dprobs, torch.float32), _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                   _ptr(dev_status, torch.int32, "dev_status"),
                   None if weight_cache is None else _ptr(weight_cache.buffer, torch.uint8, "weight_cache"),
                   0 if weight_cache is None else weight_cache.buffer.numel(),
                   _ptr(mg_gu, torch.float32, "main_grad_gate_up"), _ptr(mg_d, torch.float32, "main_grad_down"))
    name = "mxg_grouped_mlp_bf16_bwd" if bf16 else ("mxg_grouped_mlp_fp8_bwd" if fp8 else "mxg_grouped_mlp_bwd")
    if stage is None:
        _check(name, getattr(lib(), name)(ctypes.byref(a), _stream(stream)))
    else:
        _check(name + "_stage", getattr(lib(), name + "_stage")(ctypes.byref(a), stage, _stream(stream)))
    if main_grad is not None:
        return dx, mg_gu, mg_d, dprobs
    return dx, dw_gate_up, dw_down, dprobs


def mxg_bench_mxfp8_mma_peak(steps: int, dev_status: torch.Tensor, stream=None) -> float:
    """Enqueue the MXFP8 MMA-only peak loop; returns the launch's flop count
    (time it with events on the same stream)."""
    flops = ctypes.c_double(0.0)
    _check("mxg_bench_mxfp8_mma_peak", lib().mxg_bench_mxfp8_mma_peak(
        int(steps), ctypes.byref(flops), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return float(flops.value)


def mxg_mxfp8_grouped_rows_capacity(rows: int, groups: int, layout: int = MXG_LAYOUT_CANONICAL) -> int:
    return int(lib().mxg_mxfp8_grouped_rows_capacity(rows, groups, layout))


def mxg_mxfp8_quantize_grouped(x: torch.Tensor, group_offsets: torch.Tensor, dev_status: torch.Tensor,
                               row: bool = True, col: bool = True, layout: int = MXG_LAYOUT_CANONICAL,
                               stream=None) -> dict:
    """x bf16 [rows, cols] in groups (group_offsets int32 [groups+1]) -> the
    padded group layout: 'padded_offsets', and 'q_row','s_row' / 'q_col','s_col'."""
    rows, cols = x.shape
    groups = group_offsets.numel() - 1
    cap = mxg_mxfp8_grouped_rows_capacity(rows, groups, layout)
    if cap == 0:
        raise ValueError(f"unsupported grouped quantisation rows={rows} groups={groups}")
    dev = x.device
    out = {"padded_offsets": torch.empty(groups + 1, dtype=torch.int32, device=dev), "capacity": cap}
    if row:
        out["q_row"] = torch.empty((cap, cols), dtype=torch.uint8, device=dev)
        out["s_row"] = torch.empty(cap * cols // 32, dtype=torch.uint8, device=dev)
    if col:
        out["q_col"] = torch.empty((cols, cap), dtype=torch.uint8, device=dev)
        out["s_col"] = torch.empty(cap * cols // 32, dtype=torch.uint8, device=dev)
    _check("mxg_mxfp8_quantize_grouped", lib().mxg_mxfp8_quantize_grouped(
        _ptr(_bits(x), None, "x"), rows, cols, _ptr(group_offsets, torch.int32, "group_offsets"), groups,
        _ptr(out["padded_offsets"]), _ptr(out.get("q_row")), _ptr(out.get("s_row")), _ptr(out.get("q_col")),
        _ptr(out.get("s_col")), layout, _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return out


def mxg_gather_rows(src: torch.Tensor, index: torch.Tensor, dev_status: torch.Tensor, div: int = 1,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[r] = src[index[r] // div] (rows of src's trailing dimensions)."""
    src_rows = src.shape[0]
    row_bytes = src[0].numel() * src.element_size() if src.dim() > 1 else src.element_size()
    rows = index.numel()
    out = torch.empty((rows,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device) if out is None else out
    _check("mxg_gather_rows", lib().mxg_gather_rows(
        _ptr(src, None, "src"), src_rows, row_bytes, _ptr(index, torch.int32, "index"), div, rows,
        _ptr(out, src.dtype, "out"), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return out


def mxg_combine(rows: torch.Tensor, row_of_src: torch.Tensor, k: int, dev_status: torch.Tensor,
                y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j rows[row_of_src[t*k + j]] (fp32 sum in slot order, bf16 out)."""
    src_rows, H = rows.shape
    T = row_of_src.numel() // k
    y = torch.empty((T, H), dtype=torch.bfloat16, device=rows.device) if y is None else y
    _check("mxg_combine", lib().mxg_combine(
        _ptr(_bits(rows), torch.int16, "rows"), src_rows, _ptr(row_of_src, torch.int32, "row_of_src"), T, k, H,
        _ptr(_bits(y), torch.int16, "y"), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return y


def mxg_mlp_grouped_saved_bytes(R, H, I, E) -> int:
    return int(lib().mxg_mlp_grouped_saved_bytes(R, H, I, E))


def mxg_mlp_grouped_workspace_bytes(R, H, I, E) -> int:
    return int(lib().mxg_mlp_grouped_workspace_bytes(R, H, I, E))


def mxg_grouped_mlp_fwd_grouped(x, split_sizes, probs, w_gate_up, w_down, saved, workspace, dev_status, y=None,
                                save_for_backward: bool = True, weight_cache: WeightCache | None = None,
                                stream=None):
    """Forward on rows already grouped by expert (split_sizes int32 [E] on the
    device, probs fp32 [R]); returns the per-row outputs y [R, H]."""
    R, H = x.shape
    if weight_cache is not None:
        E, I = weight_cache.E, weight_cache.I
    else:
        E, N2, _ = w_gate_up.shape
        I = N2 // 2
    y = torch.empty((R, H), dtype=torch.bfloat16, device=x.device) if y is None else y
    a = MlpGroupedFwdArgs(R, H, I, E, _ptr(_bits(x), torch.int16, "x"), _ptr(split_sizes, torch.int32, "split_sizes"),
                          _ptr(probs, torch.float32, "probs"), _ptr(_bits(w_gate_up), torch.int16, "w_gate_up"),
                          _ptr(_bits(w_down), torch.int16, "w_down"), _ptr(_bits(y), torch.int16, "y"),
                          _ptr(saved, torch.uint8, "saved"), saved.numel(), _ptr(workspace, torch.uint8, "workspace"),
                          workspace.numel(), 1 if save_for_backward else 0,
                          _ptr(dev_status, torch.int32, "dev_status"),
                          None if weight_cache is None else _ptr(weight_cache.buffer, torch.uint8, "weight_cache"),
                          0 if weight_cache is None else weight_cache.buffer.numel())
    _check("mxg_grouped_mlp_fwd_grouped", lib().mxg_grouped_mlp_fwd_grouped(ctypes.byref(a), _stream(stream)))
    return y


def mxg_router_fwd_permute(x: torch.Tensor, w_router: torch.Tensor, k: int, dev_status: torch.Tensor, stream=None):
    """Router logits + route + permute in one call; returns (logits, ids,
    probs, permute dict as mxg_route_permute)."""
    T, H = x.shape
    E = w_router.shape[0]
    dev = x.device
    logits = torch.empty((T, E), dtype=torch.float32, device=dev)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    probs = torch.empty((T, k), dtype=torch.float32, device=dev)
    ws_bytes = int(lib().mxg_route_permute_workspace_bytes(T, k, E))
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    out = {"split_sizes": torch.empty(E, dtype=torch.int32, device=dev),
           "src_of_row": torch.empty(T * k, dtype=torch.int32, device=dev),
           "row_of_src": torch.empty(T * k, dtype=torch.int32, device=dev),
           "padded_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev)}
    _check("mxg_router_fwd_permute", lib().mxg_router_fwd_permute(
        _ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.bfloat16, "w_router"), T, H, E, k,
        _ptr(logits), _ptr(ids), _ptr(probs), _ptr(out["split_sizes"]), _ptr(out["src_of_row"]),
        _ptr(out["row_of_src"]), _ptr(out["padded_offsets"]), _ptr(ws), ws_bytes,
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))
    return logits, ids, probs, out


def mxg_grouped_mlp_fwd_grouped_mx(xq, xs, split_sizes, probs, w_gate_up, w_down, saved, workspace, dev_status,
                                   H: int, y=None, weight_cache: WeightCache | None = None, stream=None):
    """Inference forward on grouped rows given as row-wise MXFP8: codes xq uint8
    [R, H] and canonical scales xs uint8 [R, H/32]; returns y [R, H]."""
    R = xq.shape[0]
    if weight_cache is not None:
        E, I = weight_cache.E, weight_cache.I
    else:
        E, N2, _ = w_gate_up.shape
        I = N2 // 2
    y = torch.empty((R, H), dtype=torch.bfloat16, device=xq.device) if y is None else y
    a = MlpGroupedFwdMxArgs(R, H, I, E, _ptr(xq, torch.uint8, "xq"), _ptr(xs, torch.uint8, "xs"),
                            _ptr(split_sizes, torch.int32, "split_sizes"), _ptr(probs, torch.float32, "probs"),
                            _ptr(_bits(w_gate_up), torch.int16, "w_gate_up"), _ptr(_bits(w_down), torch.int16, "w_down"),
                            _ptr(_bits(y), torch.int16, "y"), _ptr(saved, torch.uint8, "saved"), saved.numel(),
                            _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                            _ptr(dev_status, torch.int32, "dev_status"),
                            None if weight_cache is None else _ptr(weight_cache.buffer, torch.uint8, "weight_cache"),
                            0 if weight_cache is None else weight_cache.buffer.numel())
    _check("mxg_grouped_mlp_fwd_grouped_mx", lib().mxg_grouped_mlp_fwd_grouped_mx(ctypes.byref(a), _stream(stream)))
    return y
