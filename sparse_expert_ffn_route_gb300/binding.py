"""Thin ctypes binding of libmoe.so (include/moe.h): argument marshalling only.

Every function takes CUDA torch tensors, passes their device pointers and the
current CUDA stream to the C entry point of the same name, and raises
``MoeError`` with the library's message on a nonzero return code.  All the
layer's arithmetic runs in the library's kernels; there is no other code path.
If libmoe.so is missing, loading raises ``ImportError``.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_ARG = -1
MOE_ERR_SHAPE = -2
MOE_ERR_ALIGN = -3
MOE_ERR_CUDA = -4
MOE_ERR_TIMEOUT = -5
MOE_ERR_UNSUPPORTED = -6
MOE_ERR_WORKSPACE = -7
MOE_ERR_DEVICE = -8
MOE_FLAG_SYNC_CHECK = 1
MOE_FLAG_STAGE_EVENTS = 2
MOE_FFN_WARP_GEMV = 0
MOE_FFN_TENSOR = 1
MOE_FFN_ROW_GEMV = 2
MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1
MOE_DTYPE_F16 = 2
MOE_GATE_NONE = 0
MOE_GATE_CHANNEL = 1
MOE_GATE_TOKEN = 2
MOE_GATE_FULL = 3
STAGES = ("router", "select", "permute", "plan", "quant", "gate_up", "quant_h", "down", "combine")

# every symbol include/moe.h declares
EXPORTS = ("moe_workspace_size", "moe_route", "moe_permute", "moe_expert_ffn", "moe_combine",
           "moe_layer_forward", "moe_check_errors", "moe_stage_times", "moe_last_error_string",
           "moe_route_noalloc", "moe_ffn_uses_tensor_cores", "moe_route_lookahead",
           "moe_topk_hits", "moe_quantize_int4_gs64", "moe_quantize_int3_g64",
           "moe_selftest_wait_timeout",
           "moe_layer_forward_host", "moe_ffn_path", "moe_ffn_path_down",
           "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_mxfp4_matmul", "moe_mxfp4_expert_ffn",
           "moe_mxfp4_workspace_size", "moe_gated_forward", "moe_gated_backward",
           "moe_gated_workspace_size", "moe_block_norm_forward", "moe_block_norm_backward",
           "moe_block_norm_workspace_size", "moe_balance_forward", "moe_balance_backward",
           "moe_balance_workspace_size", "moe_adapter_matmul", "moe_adapter_workspace_size")


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__("%s failed (%d): %s" % (where, code, msg))
        self.code = code


class MoeConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("d_ff_shared", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("norm_topk_prob", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float), ("top_p", ctypes.c_float)]

    @classmethod
    def make(cls, hidden, n_experts, top_k, d_ff, n_shared=0, d_ff_shared=0, norm_topk_prob=1,
             routed_scaling_factor=1.0, top_p=0.0, group_size=64) -> "MoeConfig":
        return cls(hidden, n_experts, top_k, d_ff, n_shared, d_ff_shared, group_size,
                   norm_topk_prob, routed_scaling_factor, top_p)


class ExpertWeights(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("s_gate", ctypes.c_void_p),
                ("w_up", ctypes.c_void_p), ("s_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("s_down", ctypes.c_void_p)]

    @classmethod
    def of(cls, d: Dict[str, torch.Tensor]) -> "ExpertWeights":
        return cls(*[_ptr(d[k]) for k in ("w_gate", "s_gate", "w_up", "s_up", "w_down", "s_down")])


class ExpertMxfp4(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("s_gate", ctypes.c_void_p),
                ("w_up", ctypes.c_void_p), ("s_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("s_down", ctypes.c_void_p)]


class FfnProbe(ctypes.Structure):
    _fields_ = [("acc_gate", ctypes.c_void_p), ("acc_up", ctypes.c_void_p),
                ("acc_down", ctypes.c_void_p), ("hq", ctypes.c_void_p),
                ("h_scale", ctypes.c_void_p)]


class Routing(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("w", ctypes.c_void_p), ("keff", ctypes.c_void_p)]


_lib = None


def load_library():
    """Load libmoe.so (ImportError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY_PATH):
        raise ImportError("libmoe.so not found at %s; build it with "
                          "`python -m sparse_expert_ffn_route_gb300.build`" % LIBRARY_PATH)
    L = ctypes.CDLL(LIBRARY_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.moe_workspace_size.argtypes = [vp, i32]
    L.moe_workspace_size.restype = sz
    L.moe_ffn_uses_tensor_cores.argtypes = [vp, i32]
    L.moe_ffn_uses_tensor_cores.restype = i32
    L.moe_ffn_path.argtypes = [vp, i32]
    L.moe_ffn_path.restype = i32
    L.moe_ffn_path_down.argtypes = [vp, i32]
    L.moe_ffn_path_down.restype = i32
    L.moe_route.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    L.moe_route_lookahead.argtypes = [vp, vp, vp, ctypes.c_float, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    L.moe_topk_hits.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp]
    L.moe_quantize_int4_gs64.argtypes = [vp, i32, i32, vp, vp, vp]
    L.moe_quantize_int3_g64.argtypes = [vp, i32, i32, vp, vp, vp]
    L.moe_selftest_wait_timeout.argtypes = [vp, sz, i32, vp]
    L.moe_permute.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_expert_ffn.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_combine.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    L.moe_layer_forward.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, i32, vp]
    L.moe_layer_forward_host.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, i32, vp]
    L.moe_check_errors.argtypes = [vp, sz, vp]
    L.moe_stage_times.argtypes = [vp, vp, i32]
    L.moe_route_noalloc.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp]
    i64 = ctypes.c_longlong
    L.moe_quantize_mxfp4.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp]
    L.moe_dequantize_mxfp4.argtypes = [vp, vp, i64, i32, vp, i32, vp]
    L.moe_mxfp4_matmul.argtypes = [vp, vp, i32, vp, vp, i32, vp, i32, i32, vp, i32, vp, sz, vp]
    L.moe_mxfp4_expert_ffn.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, i32, vp, sz, vp]
    L.moe_mxfp4_workspace_size.argtypes = [vp, i32]
    L.moe_mxfp4_workspace_size.restype = sz
    L.moe_gated_forward.argtypes = [vp, i64, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.moe_gated_backward.argtypes = [vp, vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp,
                                     sz, vp]
    L.moe_gated_workspace_size.argtypes = [i32, i32, i32, i32]
    L.moe_gated_workspace_size.restype = sz
    f32 = ctypes.c_float
    L.moe_block_norm_forward.argtypes = [vp, i64, i32, vp, i64, vp, i32, i32, vp, vp, f32, f32, f32, i32, i32, vp, vp, vp, vp]
    L.moe_block_norm_backward.argtypes = [vp, i64, i32, vp, i64, vp, i32, i32, vp, vp, vp, f32, f32, i32, i32, vp, vp, vp, vp,
                                          vp, vp, vp, vp, sz, vp]
    L.moe_block_norm_workspace_size.argtypes = [i32, i32]
    L.moe_block_norm_workspace_size.restype = sz
    L.moe_balance_forward.argtypes = [vp, vp, i32, i64, vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    L.moe_balance_backward.argtypes = [vp, vp, i32, i64, vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp]
    L.moe_balance_workspace_size.argtypes = [vp, i32, i32]
    L.moe_balance_workspace_size.restype = sz
    L.moe_adapter_matmul.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, vp, i32, vp, sz, vp]
    L.moe_adapter_workspace_size.argtypes = [i32, i32]
    L.moe_adapter_workspace_size.restype = sz
    L.moe_last_error_string.argtypes = []
    L.moe_last_error_string.restype = ctypes.c_char_p
    _lib = L
    return L


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where, load_library().moe_last_error_string().decode())


def last_error() -> str:
    return load_library().moe_last_error_string().decode()


def moe_workspace_size(cfg: MoeConfig, max_tokens: int) -> int:
    return int(load_library().moe_workspace_size(ctypes.byref(cfg), max_tokens))


def moe_ffn_uses_tensor_cores(cfg: MoeConfig, T: int) -> int:
    """1 if a call with T tokens runs the tensor-core grouped GEMM, 0 for the GEMV kernels,
    -1 for an invalid config or T."""
    return int(load_library().moe_ffn_uses_tensor_cores(ctypes.byref(cfg), T))


def moe_ffn_path(cfg: MoeConfig, T: int) -> int:
    """The grouped expert-FFN kernel a call with T tokens runs for gate/up:
    MOE_FFN_WARP_GEMV, MOE_FFN_TENSOR or MOE_FFN_ROW_GEMV; -1 for an invalid config or T."""
    return int(load_library().moe_ffn_path(ctypes.byref(cfg), T))


def moe_ffn_path_down(cfg: MoeConfig, T: int) -> int:
    """The same for the down projection."""
    return int(load_library().moe_ffn_path_down(ctypes.byref(cfg), T))


def alloc_workspace(cfg: MoeConfig, max_tokens: int, device="cuda") -> torch.Tensor:
    """Zeroed device workspace for up to ``max_tokens`` tokens (uint8 tensor)."""
    n = moe_workspace_size(cfg, max_tokens)
    if n == 0:
        raise MoeError(MOE_ERR_SHAPE, "moe_workspace_size", "invalid config or token count")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_route(cfg, x, w_router, bias, ids, w, keff, workspace, stream=None):
    T = x.shape[0]
    _check(load_library().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(w_router), _ptr(bias), T,
                                     _ptr(ids), _ptr(w), _ptr(keff), _ptr(workspace),
                                     workspace.numel(), _stream(stream)), "moe_route")


def moe_route_lookahead(cfg, x, norm_w, eps, w_router, bias, ids, w, keff, workspace, stream=None):
    """A layer's top-K predicted from the residual state x: RMSNorm with norm_w and eps, then
    the layer's router (w_router, bias); outputs as moe_route."""
    T = x.shape[0]
    _check(load_library().moe_route_lookahead(ctypes.byref(cfg), _ptr(x), _ptr(norm_w), float(eps),
                                               _ptr(w_router), _ptr(bias), T, _ptr(ids), _ptr(w),
                                               _ptr(keff), _ptr(workspace), workspace.numel(),
                                               _stream(stream)), "moe_route_lookahead")


def moe_topk_hits(cfg, ids_pred, keff_pred, ids_true, keff_true, hits, stream=None):
    """Per token, how many experts the predicted and the true routing both keep."""
    T = keff_pred.shape[0]
    _check(load_library().moe_topk_hits(ctypes.byref(cfg), _ptr(ids_pred), _ptr(keff_pred),
                                         _ptr(ids_true), _ptr(keff_true), T, _ptr(hits),
                                         _stream(stream)), "moe_topk_hits")


def moe_quantize_int3_g64(w, packed, scales, stream=None):
    """fp32 weights w [rows][K] (K a multiple of 64) -> int3-g64: packed [rows][3K/8] uint8
    and scales [rows][K/64] float32 (every leading dimension flattened into rows)."""
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    _check(load_library().moe_quantize_int3_g64(_ptr(w), rows, K, _ptr(packed), _ptr(scales),
                                                 _stream(stream)), "moe_quantize_int3_g64")


def moe_quantize_int4_gs64(w, packed, scales, stream=None):
    """fp32 weights w [rows][K] (K a multiple of 64) -> int4-gs64: packed [rows][K/2] uint8
    and scales [rows][K/64] float32 (every leading dimension flattened into rows)."""
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    _check(load_library().moe_quantize_int4_gs64(_ptr(w), rows, K, _ptr(packed), _ptr(scales),
                                                  _stream(stream)), "moe_quantize_int4_gs64")


def moe_selftest_wait_timeout(workspace, polls: int = 4096, stream=None):
    """Make one bounded device wait run out on purpose; moe_check_errors then reports
    MOE_ERR_TIMEOUT (the error path of the kernels' waits, with no fault or hang)."""
    _check(load_library().moe_selftest_wait_timeout(_ptr(workspace), workspace.numel(), int(polls),
                                                     _stream(stream)), "moe_selftest_wait_timeout")


def moe_route_noalloc(cfg, x, w_router, bias, ids, w, keff, stream=None):
    """moe_route without a workspace (the router scratch is a fixed array inside libmoe.so,
    so the call allocates nothing); same outputs as moe_route, batches up to its limit."""
    T = x.shape[0]
    _check(load_library().moe_route_noalloc(ctypes.byref(cfg), _ptr(x), _ptr(w_router),
                                             _ptr(bias), T, _ptr(ids), _ptr(w), _ptr(keff),
                                             _stream(stream)), "moe_route_noalloc")


def moe_permute(cfg, ids, keff, counts, offsets, tok, slot, uniq, n_uniq, workspace, stream=None):
    T = keff.shape[0]
    _check(load_library().moe_permute(ctypes.byref(cfg), _ptr(ids), _ptr(keff), T, _ptr(counts),
                                       _ptr(offsets), _ptr(tok), _ptr(slot), _ptr(uniq),
                                       _ptr(n_uniq), _ptr(workspace), workspace.numel(),
                                       _stream(stream)), "moe_permute")


def moe_expert_ffn(cfg, x, routed: Dict[str, torch.Tensor], offsets, tok, uniq, n_uniq, y_pairs,
                   workspace, probe: Optional[Dict[str, torch.Tensor]] = None, stream=None):
    T = x.shape[0]
    rw = ExpertWeights.of(routed)
    pr = None
    if probe is not None:
        pr = FfnProbe(*[_ptr(probe.get(k)) for k in ("acc_gate", "acc_up", "acc_down", "hq",
                                                       "h_scale")])
    _check(load_library().moe_expert_ffn(ctypes.byref(cfg), _ptr(x), T, ctypes.byref(rw),
                                          _ptr(offsets), _ptr(tok), _ptr(uniq), _ptr(n_uniq),
                                          _ptr(y_pairs), ctypes.byref(pr) if pr else None,
                                          _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_expert_ffn")


def moe_combine(cfg, y_pairs, ids, keff, w, offsets, tok, y, workspace, x=None,
                shared: Optional[Dict[str, torch.Tensor]] = None, stream=None):
    T = keff.shape[0]
    sw = ExpertWeights.of(shared) if shared is not None else None
    _check(load_library().moe_combine(ctypes.byref(cfg), _ptr(y_pairs), _ptr(ids), _ptr(keff),
                                       _ptr(w), _ptr(offsets), _ptr(tok), T, _ptr(x),
                                       ctypes.byref(sw) if sw else None, _ptr(y),
                                       _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_combine")


def moe_layer_forward(cfg, x, w_router, bias, routed, shared, y, workspace, routing=None,
                      flags: int = 0, stream=None):
    T = x.shape[0]
    rw = ExpertWeights.of(routed)
    sw = ExpertWeights.of(shared) if shared is not None else None
    ro = None
    if routing is not None:
        ro = Routing(_ptr(routing.get("ids")), _ptr(routing.get("w")), _ptr(routing.get("keff")))
    _check(load_library().moe_layer_forward(ctypes.byref(cfg), _ptr(x), T, _ptr(w_router),
                                             _ptr(bias), ctypes.byref(rw),
                                             ctypes.byref(sw) if sw else None, _ptr(y),
                                             ctypes.byref(ro) if ro else None, _ptr(workspace),
                                             workspace.numel(), flags, _stream(stream)),
           "moe_layer_forward")


def moe_layer_forward_host(cfg, x_host, w_router, bias, routed, shared, y_host, workspace,
                           routing=None, flags: int = 0, stream=None):
    """moe_layer_forward on host tensors x_host / y_host (CPU, pinned for asynchronous
    copies): the library copies x in, runs the layer and copies y out on the stream."""
    if x_host.is_cuda or y_host.is_cuda:
        raise ValueError("moe_layer_forward_host takes CPU tensors for x and y")
    T = x_host.shape[0]
    rw = ExpertWeights.of(routed)
    sw = ExpertWeights.of(shared) if shared is not None else None
    ro = None
    if routing is not None:
        ro = Routing(_ptr(routing.get("ids")), _ptr(routing.get("w")), _ptr(routing.get("keff")))
    _check(load_library().moe_layer_forward_host(ctypes.byref(cfg), _ptr(x_host), T, _ptr(w_router),
                                                  _ptr(bias), ctypes.byref(rw),
                                                  ctypes.byref(sw) if sw else None, _ptr(y_host),
                                                  ctypes.byref(ro) if ro else None, _ptr(workspace),
                                                  workspace.numel(), flags, _stream(stream)),
           "moe_layer_forward_host")


def moe_check_errors(workspace, stream=None):
    _check(load_library().moe_check_errors(_ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_check_errors")


def moe_stage_times(reset: bool = True):
    """Per-stage device milliseconds and kernel launches of the layer calls made with
    MOE_FLAG_STAGE_EVENTS on this thread since the last reset: {stage: (ms, launches)}."""
    ms = (ctypes.c_double * len(STAGES))()
    n = (ctypes.c_longlong * len(STAGES))()
    _check(load_library().moe_stage_times(ms, n, 1 if reset else 0), "moe_stage_times")
    return {name: (ms[i], int(n[i])) for i, name in enumerate(STAGES)}


# --- MXFP4 and the 16-bit gated block ----------------------------------------------------
# These check what the C entry points cannot see: types, shapes, strides and devices of the tensors.
# Each of them takes its first tensor's device, which has to be the current one (the library launches
# there), and asks for the others, the workspace among them, on the same.
# (not a public name: a torch without it takes the public way, at 2.9 us a call for 0.1)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = torch.cuda.current_device
_device_count = functools.lru_cache(maxsize=None)(torch.cuda.device_count)


def _raw_stream(stream, device: int) -> int:
    """The handle of `stream`, or of the current stream of the device (without the Stream object that
    torch.cuda.current_stream makes, where a one-token call takes 5 us)."""
    return _current_stream(device) if stream is None else stream.cuda_stream


_DTYPES = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16}


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32, bfloat16 or float16 (got %s)" % (name, t.dtype))
    return code


def _dense(t: torch.Tensor, name: str, shape, dtype, device: int) -> int:
    """Device pointer of a contiguous tensor of the given shape and type on `device`."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    raise ValueError("%s must be a contiguous CUDA tensor %s of %s on device %d (got %s of %s on %s%s)" % (
        name, tuple(shape), dtype, device, tuple(t.shape), t.dtype, t.device, "" if t.is_contiguous() else ", strided"))


def _space(t: torch.Tensor, device: int) -> int:
    """Device pointer of a workspace: contiguous bytes on `device`."""
    if t.dtype is torch.uint8 and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    raise ValueError("the workspace must be a contiguous CUDA tensor of torch.uint8 on device %d (got %s on %s%s)" % (
        device, t.dtype, t.device, "" if t.is_contiguous() else ", strided"))


def _device(t: torch.Tensor, name: str) -> int:
    """The index of t's device, which has to be the current CUDA device."""
    device = t.get_device()
    if device < 0:
        raise ValueError("%s must be a contiguous CUDA tensor (got one on %s)" % (name, t.device))
    if _device_count() > 1 and device != _current_device():
        raise ValueError("%s is on device %d, the current device is %d" % (name, device, _current_device()))
    return device


def _rows(t: torch.Tensor, name: str):
    """(device, rows, width, row stride) of a 2-D CUDA tensor whose rows are contiguous."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be a 2-D CUDA tensor" % name)
    device = _device(t, name)
    rows, width = shape
    if t.is_contiguous():
        return device, rows, width, width
    if width > 1 and t.stride(1) != 1:
        raise ValueError("rows of %s must be contiguous" % name)
    return device, rows, width, t.stride(0)


def moe_quantize_mxfp4(x, codes, scales, stream=None):
    """Rows x [rows][K] (float32, bfloat16 or float16; K a multiple of 32, rows may be strided)
    -> MXFP4: codes [rows][K/2] uint8 and scales [rows][K/32] uint8.  A contiguous x of more
    dimensions is taken as its rows laid end to end."""
    if len(x.shape) > 2 and x.is_contiguous():
        x = x.view(-1, x.shape[-1])
        codes, scales = codes.view(-1, codes.shape[-1]), scales.view(-1, scales.shape[-1])
    dev, rows, K, ld = _rows(x, "x")
    rc = load_library().moe_quantize_mxfp4(
        x.data_ptr(), _dtype(x, "x"), ld, rows, K, _dense(codes, "codes", (rows, K // 2), torch.uint8, dev),
        _dense(scales, "scales", (rows, K // 32), torch.uint8, dev), _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_quantize_mxfp4")


def moe_dequantize_mxfp4(codes, scales, y, stream=None):
    """The values that MXFP4 codes [..][K/2] and scales [..][K/32] stand for, into y [..][K]."""
    shape, dev = y.shape, _device(y, "y")
    if len(shape) == 2:
        rows, K = shape
        c, sc = (rows, K // 2), (rows, K // 32)
    else:
        K, lead = shape[-1], tuple(shape[:-1])
        rows, c, sc = (y.numel() // K if K else 0), lead + (K // 2,), lead + (K // 32,)
    rc = load_library().moe_dequantize_mxfp4(
        _dense(codes, "codes", c, torch.uint8, dev), _dense(scales, "scales", sc, torch.uint8, dev), rows, K,
        _dense(y, "y", shape, y.dtype, dev), _dtype(y, "y"), _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_dequantize_mxfp4")


def alloc_mxfp4_matmul_workspace(device="cuda") -> torch.Tensor:
    """Zeroed workspace of moe_mxfp4_matmul (the error word)."""
    return torch.zeros(256, dtype=torch.uint8, device=device)


def moe_mxfp4_matmul(x, x_scales, w, w_scales, y, workspace, offsets=None, stream=None):
    """y [rows][N] = x w^T by group: x [rows][K/2], x_scales [rows][K/32]; w [groups][N][K/2] (or
    [N][K/2]), w_scales alike; offsets [groups + 1] int32 (None: one group, all rows)."""
    rows, half = x.shape
    K32, u8, dev = half // 16, torch.uint8, _device(x, "x")
    if w.dim() == 2:
        groups, N = 1, w.shape[0]
        pw, psw = _dense(w, "w", (N, half), u8, dev), _dense(w_scales, "w_scales", (N, K32), u8, dev)
    else:
        groups, N = w.shape[0], w.shape[1]
        pw, psw = _dense(w, "w", (groups, N, half), u8, dev), _dense(w_scales, "w_scales", (groups, N, K32), u8, dev)
    _check(load_library().moe_mxfp4_matmul(
        _dense(x, "x", (rows, half), u8, dev), _dense(x_scales, "x_scales", (rows, K32), u8, dev), rows, pw, psw, groups,
        None if offsets is None else _dense(offsets, "offsets", (groups + 1,), torch.int32, dev), N, 2 * half,
        _dense(y, "y", (rows, N), y.dtype, dev), _dtype(y, "y"), _space(workspace, dev), workspace.numel(),
        _raw_stream(stream, dev)), "moe_mxfp4_matmul")


def moe_mxfp4_workspace_size(cfg: MoeConfig, max_tokens: int) -> int:
    return int(load_library().moe_mxfp4_workspace_size(ctypes.byref(cfg), max_tokens))


def alloc_mxfp4_workspace(cfg: MoeConfig, max_tokens: int, device="cuda") -> torch.Tensor:
    """Workspace of moe_mxfp4_expert_ffn for up to ``max_tokens`` tokens, its head zeroed."""
    n = moe_mxfp4_workspace_size(cfg, max_tokens)
    if n == 0:
        raise MoeError(MOE_ERR_SHAPE, "moe_mxfp4_workspace_size", "invalid config or token count")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_mxfp4_expert_ffn(cfg, x, weights: Dict[str, torch.Tensor], y_pairs, workspace, offsets=None,
                         tok=None, stream=None):
    """Routed expert FFN on MXFP4 weights: x [T][H] -> y_pairs [T * top_k][H] in the order of
    offsets / tok (as moe_permute writes them; both None: one expert, every token).  weights:
    w_gate, w_up [E][F][H/2], w_down [E][H][F/2] and s_gate, s_up [E][F][H/32],
    s_down [E][H][F/32], uint8."""
    T, H, F, E, P = x.shape[0], cfg.hidden, cfg.d_ff, cfg.n_experts, y_pairs.shape[0]
    u8, up, down, dev = torch.uint8, (E, F, H // 2), (E, H, F // 2), _device(x, "x")
    s_up, s_down = (E, F, H // 32), (E, H, F // 32)
    w = ExpertMxfp4(*[_dense(weights[k], k, shape, u8, dev) for k, shape in (
        ("w_gate", up), ("s_gate", s_up), ("w_up", up), ("s_up", s_up), ("w_down", down), ("s_down", s_down))])
    if P != T * cfg.top_k:
        raise ValueError("y_pairs must have T * top_k = %d rows (got %d)" % (T * cfg.top_k, P))
    _check(load_library().moe_mxfp4_expert_ffn(
        ctypes.byref(cfg), _dense(x, "x", (T, H), x.dtype, dev), _dtype(x, "x"), T, ctypes.byref(w),
        None if offsets is None else _dense(offsets, "offsets", (E + 1,), torch.int32, dev),
        None if tok is None else _dense(tok, "tok", (P,), torch.int32, dev),
        _dense(y_pairs, "y_pairs", (P, H), y_pairs.dtype, dev), _dtype(y_pairs, "y_pairs"),
        _space(workspace, dev), workspace.numel(), _raw_stream(stream, dev)), "moe_mxfp4_expert_ffn")


def moe_gated_workspace_size(T: int, H: int, F: int, train: bool) -> int:
    return int(load_library().moe_gated_workspace_size(T, H, F, 1 if train else 0))


def alloc_gated_workspace(T: int, H: int, F: int, train: bool, device="cuda") -> torch.Tensor:
    """Workspace of the gated block's calls for T tokens, its head zeroed."""
    n = moe_gated_workspace_size(T, H, F, train)
    if n == 0:
        raise MoeError(MOE_ERR_SHAPE, "moe_gated_workspace_size", "sizes outside the limits")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_gated_forward(x, w_gate, w_up, h, workspace, g=None, u=None, stream=None):
    """h [T][F] = silu(x w_gate^T) * (x w_up^T), all bfloat16 or all float16.  Rows of x [T][H]
    may be strided.  g, u [T][F] of the same type are filled for moe_gated_backward with the factors of dh that
    give dg and du, as 16-bit words to be handed on: they are not the values of x w_gate^T and x w_up^T."""
    dev, T, H, ld = _rows(x, "x")
    F, dt = w_gate.shape[0], x.dtype
    _check(load_library().moe_gated_forward(
        x.data_ptr(), ld, _dense(w_gate, "w_gate", (F, H), dt, dev), _dense(w_up, "w_up", (F, H), dt, dev),
        _dtype(x, "x"), T, H, F, _dense(h, "h", (T, F), dt, dev),
        None if g is None else _dense(g, "g", (T, F), dt, dev), None if u is None else _dense(u, "u", (T, F), dt, dev),
        _space(workspace, dev), workspace.numel(), _raw_stream(stream, dev)), "moe_gated_forward")


def moe_gated_backward(dh, x, w_gate, w_up, g, u, dx, dw_gate, dw_up, workspace, stream=None):
    """Gradients of moe_gated_forward from dh [T][F] and the g, u that it filled: dx [T][H] (or None) and
    dw_gate, dw_up [F][H] (or both None), written in full."""
    dev, T, H, ld = _rows(x, "x")
    F, dt = w_gate.shape[0], x.dtype
    opt = lambda t, name, shape: None if t is None else _dense(t, name, shape, dt, dev)  # noqa: E731
    _check(load_library().moe_gated_backward(
        _dense(dh, "dh", (T, F), dt, dev), x.data_ptr(), ld, _dense(w_gate, "w_gate", (F, H), dt, dev),
        _dense(w_up, "w_up", (F, H), dt, dev), _dense(g, "g", (T, F), dt, dev), _dense(u, "u", (T, F), dt, dev),
        _dtype(x, "x"), T, H, F, opt(dx, "dx", (T, H)), opt(dw_gate, "dw_gate", (F, H)),
        opt(dw_up, "dw_up", (F, H)), _space(workspace, dev), workspace.numel(),
        _raw_stream(stream, dev)), "moe_gated_backward")


# --- Around the expert layer: norms between blocks, the routing's balance, adapters ---------------------
def _strided(t: torch.Tensor, name: str, rows: int, width: int, device: int):
    """(pointer, row stride) of a 2-D tensor [rows][width] on `device` whose rows are contiguous."""
    dev, r, w, ld = _rows(t, name)
    if (r, w) != (rows, width) or dev != device:
        raise ValueError("%s must be [%d][%d] on device %d (got %s on %s)" % (
            name, rows, width, device, tuple(t.shape), t.device))
    return t.data_ptr(), ld


def _gate(gate, dgate, T: int, H: int, dtype, device: int):
    """(pointer, kind) of a gate [H] or [1][H], [T][1], or [T][H].  Of [1][H] for one token the gradient's type
    tells: a channel's is float32."""
    if gate is None:
        return None, MOE_GATE_NONE
    shape = tuple(gate.shape)
    if shape == (T, H) and not (T == 1 and dgate is not None and dgate.dtype is torch.float32 and dtype is not torch.float32):
        kind = MOE_GATE_FULL
    elif shape in ((H,), (1, H)):
        kind = MOE_GATE_CHANNEL
    elif shape == (T, 1):
        kind = MOE_GATE_TOKEN
    else:
        raise ValueError("gate must be [H], [T][1] or [T][H] for T %d, H %d (got %s)" % (T, H, shape))
    return _dense(gate, "gate", shape, dtype, device), kind


def moe_block_norm_workspace_size(T: int, H: int) -> int:
    return int(load_library().moe_block_norm_workspace_size(T, H))


def alloc_block_norm_workspace(T: int, H: int, device="cuda") -> torch.Tensor:
    """Workspace of moe_block_norm_backward for T rows of H, its head zeroed; for one call at a time."""
    n = moe_block_norm_workspace_size(T, H)
    if n == 0:
        raise MoeError(MOE_ERR_SHAPE, "moe_block_norm_workspace_size", "sizes outside the limits")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_block_norm_forward(x, eps, y=None, post_w=None, gate=None, pre_w=None, out=None, n=None, residual_scale=1.0,
                           branch_scale=1.0, kept=None, stream=None):
    """The step between two blocks: out [T][H] = residual_scale * x + branch_scale * gate * z, z = y or, with
    post_w, its RMSNorm times post_w; n = the RMSNorm of out times pre_w.  x and out are of the residual
    stream's type, y, gate and n of the blocks', each float32, bfloat16 or float16; post_w, pre_w [H] and
    kept [T][2] (for moe_block_norm_backward) float32.  gate: [H], [T][1] or [T][H].  Rows of x and y may be
    strided.  Without y, a first block's norm."""
    dev, T, H, ld = _rows(x, "x")
    f32 = torch.float32
    like = y if y is not None else n if n is not None else x
    dt = like.dtype
    py, ldy = (None, 0) if y is None else _strided(y, "y", T, H, dev)
    pg, kind = _gate(gate, None, T, H, dt, dev)
    rc = load_library().moe_block_norm_forward(
        x.data_ptr(), ld, _dtype(x, "x"), py, ldy, pg, kind, _dtype(like, "y"),
        None if post_w is None else _dense(post_w, "post_w", (H,), f32, dev),
        None if pre_w is None else _dense(pre_w, "pre_w", (H,), f32, dev), eps, residual_scale, branch_scale, T, H,
        None if out is None else _dense(out, "out", (T, H), x.dtype, dev),
        None if n is None else _dense(n, "n", (T, H), dt, dev),
        None if kept is None else _dense(kept, "kept", (T, 2), f32, dev), _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_block_norm_forward")


def moe_block_norm_backward(x, kept, workspace, y=None, post_w=None, gate=None, pre_w=None, dout=None, dn=None, dx=None, dy=None,
                            dgate=None, dpost=None, dpre=None, residual_scale=1.0, branch_scale=1.0, stream=None):
    """Gradients of moe_block_norm_forward from dout [T][H] (x's type) and dn [T][H] (y's), either None: dx (x's
    type), dy (y's), dpost, dpre [H] float32, and dgate, float32 in the gate's shape or for a gate [T][H] of its
    type.  A gradient that is None is not formed."""
    dev, T, H, ld = _rows(x, "x")
    f32 = torch.float32
    like = y if y is not None else dn if dn is not None else x
    dt = like.dtype
    py, ldy = (None, 0) if y is None else _strided(y, "y", T, H, dev)
    pg, kind = _gate(gate, dgate, T, H, dt, dev)
    pdg = None
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate without a gate")
        pdg = _dense(dgate, "dgate", tuple(gate.shape), dt if kind == MOE_GATE_FULL else f32, dev)
    rc = load_library().moe_block_norm_backward(
        x.data_ptr(), ld, _dtype(x, "x"), py, ldy, pg, kind, _dtype(like, "y"),
        None if post_w is None else _dense(post_w, "post_w", (H,), f32, dev),
        None if pre_w is None else _dense(pre_w, "pre_w", (H,), f32, dev), _dense(kept, "kept", (T, 2), f32, dev),
        residual_scale, branch_scale, T, H,
        None if dout is None else _dense(dout, "dout", (T, H), x.dtype, dev),
        None if dn is None else _dense(dn, "dn", (T, H), dt, dev),
        None if dx is None else _dense(dx, "dx", (T, H), x.dtype, dev),
        None if dy is None else _dense(dy, "dy", (T, H), dt, dev), pdg,
        None if dpost is None else _dense(dpost, "dpost", (H,), f32, dev),
        None if dpre is None else _dense(dpre, "dpre", (H,), f32, dev),
        _space(workspace, dev), workspace.numel(), _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_block_norm_backward")


def moe_balance_workspace_size(cfg: MoeConfig, max_tokens: int, max_seq: int) -> int:
    return int(load_library().moe_balance_workspace_size(ctypes.byref(cfg), max_tokens, max_seq))


def alloc_balance_workspace(cfg: MoeConfig, max_tokens: int, max_seq: int, device="cuda") -> torch.Tensor:
    """Workspace of moe_balance_forward for up to ``max_tokens`` tokens in up to ``max_seq`` sequences, its head zeroed."""
    n = moe_balance_workspace_size(cfg, max_tokens, max_seq)
    if n == 0:
        raise MoeError(MOE_ERR_SHAPE, "moe_balance_workspace_size", "invalid config or count")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _routing(cfg, logits, ids, keff, seq_offsets, valid):
    """(device, T, sequences, the operands that both directions begin with)."""
    dev, T, E, ld = _rows(logits, "logits")
    S, i32 = seq_offsets.numel() - 1, torch.int32
    if E != cfg.n_experts:
        raise ValueError("logits must have n_experts = %d columns (got %d)" % (cfg.n_experts, E))
    return dev, T, S, (ctypes.byref(cfg), logits.data_ptr(), _dtype(logits, "logits"), ld,
                       _dense(ids, "ids", (T, cfg.top_k), i32, dev), _dense(keff, "keff", (T,), i32, dev), T,
                       _dense(seq_offsets, "seq_offsets", (S + 1,), i32, dev), S,
                       None if valid is None else _dense(valid, "valid", (T,), torch.uint8, dev))


def moe_balance_forward(cfg, logits, ids, keff, seq_offsets, loss, counts, tokens, workspace, valid=None, stream=None):
    """How evenly a routing loads the experts: counts [S][E] int32 (kept pairs of each sequence and expert),
    tokens [S] int32 (counted tokens) and loss [1] float32, from the router's logits [T][E] (float32, bfloat16 or
    float16; rows may be strided) and moe_route's ids [T][K], keff [T].  seq_offsets [S + 1] int32; valid [T] uint8
    (None: all): tokens with 0 are left out, whatever their rows hold."""
    dev, T, S, operands = _routing(cfg, logits, ids, keff, seq_offsets, valid)
    rc = load_library().moe_balance_forward(
        *operands, _dense(loss, "loss", (1,), torch.float32, dev), _dense(counts, "counts", (S, cfg.n_experts), torch.int32, dev),
        _dense(tokens, "tokens", (S,), torch.int32, dev), _space(workspace, dev), workspace.numel(), _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_balance_forward")


def moe_balance_backward(cfg, logits, ids, keff, seq_offsets, counts, tokens, dlogits, workspace, dloss=None, dw=None,
                         valid=None, stream=None):
    """dlogits [T][E] (float32 or the logits' type) from dloss [1] float32, the balance loss's gradient, and dw [T][K]
    float32, that of the weights moe_route applies (either may be None).  counts and tokens as
    moe_balance_forward wrote them."""
    dev, T, S, operands = _routing(cfg, logits, ids, keff, seq_offsets, valid)
    f32, E = torch.float32, cfg.n_experts
    rc = load_library().moe_balance_backward(
        *operands, _dense(counts, "counts", (S, E), torch.int32, dev), _dense(tokens, "tokens", (S,), torch.int32, dev),
        None if dloss is None else _dense(dloss, "dloss", (1,), f32, dev),
        None if dw is None else _dense(dw, "dw", (T, cfg.top_k), f32, dev),
        _dense(dlogits, "dlogits", (T, E), dlogits.dtype, dev), _dtype(dlogits, "dlogits"), _space(workspace, dev),
        workspace.numel(), _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_balance_backward")


def moe_adapter_workspace_size(T: int, rank: int) -> int:
    return int(load_library().moe_adapter_workspace_size(T, rank))


def alloc_adapter_workspace(T: int = 32768, rank: int = 64, device="cuda") -> torch.Tensor:
    """Workspace of moe_adapter_matmul, its head zeroed.  It serves any T and rank: more rows or a higher rank
    than it is made for take more passes."""
    n = moe_adapter_workspace_size(T, rank)
    if n == 0:
        raise MoeError(MOE_ERR_SHAPE, "moe_adapter_workspace_size", "sizes outside the limits")
    n = max(n, moe_adapter_workspace_size(128, 128))     # the least that the highest rank takes
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def moe_adapter_matmul(x, down, up, scale, offsets, ids, y, workspace, base=None, stream=None):
    """y = base + scale[a] * (x down[a]^T) up[a]^T with a = ids[s] for the rows of segment s: x [T][K] (rows may be
    strided), down [A][R][K], up [A][N][R], all bfloat16 or all float16; scale [A] float32 or None; offsets [S + 1],
    ids [S] int32 (-1: no adapter); base, y [T][N] of one type, base y itself or None (zero)."""
    dev, T, K, ld = _rows(x, "x")
    dt = x.dtype
    if down.dim() != 3 or up.dim() != 3:
        raise ValueError("down must be [A][R][K] and up [A][N][R]")
    A, R, N = down.shape[0], down.shape[1], up.shape[1]
    S = ids.numel()
    rc = load_library().moe_adapter_matmul(
        x.data_ptr(), ld, _dtype(x, "x"), T, K, _dense(down, "down", (A, R, K), dt, dev), _dense(up, "up", (A, N, R), dt, dev),
        None if scale is None else _dense(scale, "scale", (A,), torch.float32, dev), A, R, N,
        _dense(offsets, "offsets", (S + 1,), torch.int32, dev), _dense(ids, "ids", (S,), torch.int32, dev), S,
        None if base is None else _dense(base, "base", (T, N), y.dtype, dev),
        _dense(y, "y", (T, N), y.dtype, dev), _dtype(y, "y"), _space(workspace, dev), workspace.numel(),
        _raw_stream(stream, dev))
    if rc:
        _check(rc, "moe_adapter_matmul")
