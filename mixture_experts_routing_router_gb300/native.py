"""ctypes binding of libmoe.so: the C-ABI calls of include/moe.h under the same
names, taking torch tensors for device buffers and the current CUDA stream.

Argument marshalling only -- every step of the layer runs in the library's
CUDA kernels.  There is no fallback: if libmoe.so is missing or cannot be
loaded, ``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_INVALID_ROUTE = 2
MOE_ERR_CAPACITY = 3
MOE_ERR_NONFINITE = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_CUDA = 6
MOE_ERR_UNSUPPORTED = 7
MOE_ERR_INTERNAL = 8

MOE_ACT_SWIGLU = 0
MOE_ACT_RELU2 = 1

MOE_TYPE_BF16 = 0
MOE_TYPE_F32 = 1

MOE_WGRAD_BF16 = 0
MOE_WGRAD_F32 = 1
MOE_WGRAD_F32_ADD = 2

# every symbol include/moe.h declares
EXPORTS = ("moe_workspace_size", "moe_workspace_init", "moe_route", "moe_dispatch", "moe_expert_up",
           "moe_expert_down", "moe_expert_ffn", "moe_combine", "moe_layer", "moe_status_read",
           "moe_status_string", "moe_last_error_message", "moe_dispatch_noalloc", "moe_gate",
           "moe_route_sigmoid", "moe_expert_up_fp8", "moe_expert_down_fp8", "moe_layer_fp8",
           "moe_expert_up_nvfp4", "moe_expert_down_nvfp4", "moe_layer_nvfp4", "moe_workspace_set_wait",
           "moe_timeout_site_read", "moe_ep_plan", "moe_layernorm", "moe_layernorm_scratch_size",
           "moe_layernorm_backward", "moe_combine_backward", "moe_dispatch_backward", "moe_route_backward",
           "moe_route_sigmoid_backward", "moe_gate_backward", "moe_expert_up_train", "moe_expert_down_backward",
           "moe_expert_up_backward", "moe_workspace_stage_size")


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = last_error_message()
        super().__init__(f"{where}: status {status} ({status_string(status)})" + (f": {msg}" if msg else ""))


class moe_shape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("inter", ctypes.c_int32), ("shared", ctypes.c_int32),
                ("shared_inter", ctypes.c_int32), ("capacity", ctypes.c_int32), ("act", ctypes.c_int32)]


def make_shape(tokens, hidden, experts, top_k, inter, act=MOE_ACT_SWIGLU, shared=0, shared_inter=0,
               capacity=0) -> moe_shape:
    return moe_shape(tokens, hidden, experts, top_k, inter, shared, shared_inter,
                     capacity if capacity > 0 else tokens, act)


def shape_of(wl) -> moe_shape:
    """moe_shape of a synth.Workload."""
    return make_shape(wl.tokens, wl.hidden, wl.experts, wl.top_k, wl.inter, wl.act, wl.shared,
                      wl.shared_inter, wl.cap)


_lock = threading.Lock()
_lib = None


def lib():
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is not built: run mixture_experts_routing_router_gb300.build.build() "
                                   "(nvcc, sm_103a); there is no CPU fallback")
            L = ctypes.CDLL(LIB_PATH)
            P, S = ctypes.c_void_p, ctypes.c_size_t
            SP = ctypes.POINTER(moe_shape)
            I32, I64 = ctypes.c_int32, ctypes.c_int64
            sig = {
                "moe_workspace_size": [SP, ctypes.POINTER(ctypes.c_size_t)],
                "moe_workspace_stage_size": [SP, ctypes.POINTER(ctypes.c_size_t)],
                "moe_workspace_init": [P, S, P],
                "moe_route": [SP, P, P, P, P, S, P],
                "moe_dispatch": [SP, P, P, P, P, P, P, P, P, S, P],
                "moe_expert_up": [SP, P, P, P, P, P, P, P, S, P],
                "moe_expert_down": [SP, P, P, P, P, P, P, P, S, P],
                "moe_expert_ffn": [SP, P, P, P, P, P, P, P, P, P, P, P, S, P],
                "moe_combine": [SP, P, P, P, P, P, P, P, S, P],
                "moe_layer": [SP, P, P, P, P, P, P, P, P, P, P, P, S, P],
                "moe_status_read": [P, P, ctypes.POINTER(ctypes.c_int)],
                "moe_dispatch_noalloc": [SP, P, P, P, P, P, P, P, P, P],
                "moe_gate": [SP, P, P, P, P, S, P],
                "moe_route_sigmoid": [SP, P, P, ctypes.c_float, P, P, P, S, P],
                "moe_expert_up_fp8": [SP, P, P, P, P, P, P, S, P],
                "moe_expert_down_fp8": [SP, P, P, P, P, P, P, S, P],
                "moe_layer_fp8": [SP, P, P, P, P, P, P, P, P, P, P, P, S, P],
                "moe_expert_up_nvfp4": [SP, P, P, P, P, P, P, P, S, P],
                "moe_expert_down_nvfp4": [SP, P, P, P, P, P, P, P, S, P],
                "moe_layer_nvfp4": [SP, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P],
                "moe_workspace_set_wait": [P, S, ctypes.c_uint64, ctypes.c_int32, P],
                "moe_timeout_site_read": [P, P, ctypes.POINTER(ctypes.c_int32)],
                "moe_ep_plan": [ctypes.c_int32] * 4 + [P] * 6,
                "moe_layernorm": [I64, I32, I32, I32, P, P, P, ctypes.c_float, P, P, P, P],
                "moe_layernorm_scratch_size": [I64, I32, ctypes.POINTER(ctypes.c_size_t)],
                "moe_layernorm_backward": [I64, I32, I32, I32] + [P] * 10 + [S, P],
                "moe_combine_backward": [SP, P, P, P, P, P, P, P, S, P],
                "moe_dispatch_backward": [SP, P, P, P, P, P, S, P],
                "moe_route_backward": [SP, P, P, P, P, P, S, P],
                "moe_route_sigmoid_backward": [SP, P, P, ctypes.c_float, P, P, P, S, P],
                "moe_gate_backward": [SP, P, P, P, P, P, P, I32, P, S, P],
                "moe_expert_up_train": [SP, P, P, P, P, P, P, S, P],
                "moe_expert_down_backward": [SP, P, P, P, P, P, P, P, I32, P, S, P],
                "moe_expert_up_backward": [SP, P, P, P, P, P, P, I32, P, S, P],
            }
            for name, args in sig.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = ctypes.c_int
            L.moe_status_string.argtypes = [ctypes.c_int]
            L.moe_status_string.restype = ctypes.c_char_p
            L.moe_last_error_message.argtypes = []
            L.moe_last_error_message.restype = ctypes.c_char_p
            _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().moe_status_string(int(status)).decode()
    except Exception:
        return "?"


def last_error_message() -> str:
    try:
        return lib().moe_last_error_message().decode()
    except Exception:
        return ""


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # the current device's current stream, without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(st, where):
    if st != MOE_OK:
        raise MoEError(st, where)


# ---- the C-ABI calls ------------------------------------------------------
def moe_workspace_size(shape: moe_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def moe_workspace_stage_size(shape: moe_shape) -> int:
    """Bytes of workspace that every call but the whole-layer ones needs."""
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_stage_size(ctypes.byref(shape), ctypes.byref(n)), "moe_workspace_stage_size")
    return n.value


WORKSPACE_HEADER = 4096       # bytes at a workspace's start that stay between calls


def moe_workspace_init(ws: torch.Tensor, stream=None):
    _check(lib().moe_workspace_init(_ptr(ws), _wsb(ws), _stream(stream)), "moe_workspace_init")


def workspace(shape: moe_shape, device="cuda") -> torch.Tensor:
    """A zero-initialised workspace tensor of moe_workspace_size bytes."""
    return torch.zeros(moe_workspace_size(shape), dtype=torch.uint8, device=device)


def _wsb(ws):
    return ws.nbytes


def moe_route(shape, logits, topk_ids, topk_w, ws, stream=None):
    _check(lib().moe_route(ctypes.byref(shape), _ptr(logits), _ptr(topk_ids), _ptr(topk_w), _ptr(ws), _wsb(ws),
                           _stream(stream)), "moe_route")


def moe_gate(shape, x, w_gate, logits, ws, stream=None):
    _check(lib().moe_gate(ctypes.byref(shape), _ptr(x), _ptr(w_gate), _ptr(logits), _ptr(ws), _wsb(ws),
                          _stream(stream)), "moe_gate")


def moe_route_sigmoid(shape, logits, bias, route_scale, topk_ids, topk_w, ws, stream=None):
    _check(lib().moe_route_sigmoid(ctypes.byref(shape), _ptr(logits), _ptr(bias), float(route_scale),
                                   _ptr(topk_ids), _ptr(topk_w), _ptr(ws), _wsb(ws), _stream(stream)),
           "moe_route_sigmoid")


def moe_dispatch(shape, x, topk_ids, counts, offsets, dest, sorted_pair, x_perm, ws, stream=None):
    _check(lib().moe_dispatch(ctypes.byref(shape), _ptr(x), _ptr(topk_ids), _ptr(counts), _ptr(offsets), _ptr(dest),
                              _ptr(sorted_pair), _ptr(x_perm), _ptr(ws), _wsb(ws), _stream(stream)), "moe_dispatch")


def moe_expert_up(shape, x_perm, offsets, w13, x, ws13, h, ws, stream=None):
    _check(lib().moe_expert_up(ctypes.byref(shape), _ptr(x_perm), _ptr(offsets), _ptr(w13), _ptr(x), _ptr(ws13),
                               _ptr(h), _ptr(ws), _wsb(ws), _stream(stream)), "moe_expert_up")


def moe_expert_down(shape, h, offsets, w2, ws2, y_perm, y_shared, ws, stream=None):
    _check(lib().moe_expert_down(ctypes.byref(shape), _ptr(h), _ptr(offsets), _ptr(w2), _ptr(ws2), _ptr(y_perm),
                                 _ptr(y_shared), _ptr(ws), _wsb(ws), _stream(stream)), "moe_expert_down")


def moe_expert_ffn(shape, x_perm, offsets, w13, w2, x, ws13, ws2, h, y_perm, y_shared, ws, stream=None):
    _check(lib().moe_expert_ffn(ctypes.byref(shape), _ptr(x_perm), _ptr(offsets), _ptr(w13), _ptr(w2), _ptr(x),
                                _ptr(ws13), _ptr(ws2), _ptr(h), _ptr(y_perm), _ptr(y_shared), _ptr(ws), _wsb(ws),
                                _stream(stream)), "moe_expert_ffn")


def moe_combine(shape, y_perm, dest, topk_w, y_shared, out, ws, stream=None, residual=None):
    _check(lib().moe_combine(ctypes.byref(shape), _ptr(y_perm), _ptr(dest), _ptr(topk_w), _ptr(y_shared),
                             _ptr(residual), _ptr(out), _ptr(ws), _wsb(ws), _stream(stream)), "moe_combine")


def moe_layer(shape, logits, ids_in, w_in, x, w13, w2, ws13, ws2, out, ws, stream=None, residual=None):
    _check(lib().moe_layer(ctypes.byref(shape), _ptr(logits), _ptr(ids_in), _ptr(w_in), _ptr(x), _ptr(w13),
                           _ptr(w2), _ptr(ws13), _ptr(ws2), _ptr(residual), _ptr(out), _ptr(ws), _wsb(ws),
                           _stream(stream)), "moe_layer")


def moe_expert_up_fp8(shape, x_perm, offsets, w13, w13_scale, h, ws, stream=None):
    """Up projection with FP8 E4M3 weights (uint8 [E, up, H]) and FP32 row scales ([E, up])."""
    _check(lib().moe_expert_up_fp8(ctypes.byref(shape), _ptr(x_perm), _ptr(offsets), _ptr(w13), _ptr(w13_scale),
                                   _ptr(h), _ptr(ws), _wsb(ws), _stream(stream)), "moe_expert_up_fp8")


def moe_expert_down_fp8(shape, h, offsets, w2, w2_scale, y_perm, ws, stream=None):
    """Down projection with FP8 E4M3 weights (uint8 [E, H, I]) and FP32 row scales ([E, H])."""
    _check(lib().moe_expert_down_fp8(ctypes.byref(shape), _ptr(h), _ptr(offsets), _ptr(w2), _ptr(w2_scale),
                                     _ptr(y_perm), _ptr(ws), _wsb(ws), _stream(stream)), "moe_expert_down_fp8")


def moe_layer_fp8(shape, logits, ids_in, w_in, x, w13, w13_scale, w2, w2_scale, out, ws, stream=None,
                  residual=None):
    """The layer with FP8 E4M3 expert weights (no shared experts)."""
    _check(lib().moe_layer_fp8(ctypes.byref(shape), _ptr(logits), _ptr(ids_in), _ptr(w_in), _ptr(x), _ptr(w13),
                               _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(residual), _ptr(out), _ptr(ws),
                               _wsb(ws), _stream(stream)), "moe_layer_fp8")


def moe_expert_up_nvfp4(shape, x_perm, offsets, w13, w13_bscale, w13_scale, h, ws, stream=None):
    """Up projection with NVFP4 weights: codes uint8 [E, up, H/2], E4M3 block
    scales uint8 [E, up, 16*ceil(H/256)], FP32 row scales [E, up]."""
    _check(lib().moe_expert_up_nvfp4(ctypes.byref(shape), _ptr(x_perm), _ptr(offsets), _ptr(w13), _ptr(w13_bscale),
                                     _ptr(w13_scale), _ptr(h), _ptr(ws), _wsb(ws), _stream(stream)),
           "moe_expert_up_nvfp4")


def moe_expert_down_nvfp4(shape, h, offsets, w2, w2_bscale, w2_scale, y_perm, ws, stream=None):
    """Down projection with NVFP4 weights: codes uint8 [E, H, I/2], block
    scales uint8 [E, H, 16*ceil(I/256)], FP32 row scales [E, H]."""
    _check(lib().moe_expert_down_nvfp4(ctypes.byref(shape), _ptr(h), _ptr(offsets), _ptr(w2), _ptr(w2_bscale),
                                       _ptr(w2_scale), _ptr(y_perm), _ptr(ws), _wsb(ws), _stream(stream)),
           "moe_expert_down_nvfp4")


def moe_layer_nvfp4(shape, logits, ids_in, w_in, x, w13, w13_bscale, w13_scale, w2, w2_bscale, w2_scale, out, ws,
                    stream=None, residual=None):
    """The layer with NVFP4 expert weights (no shared experts)."""
    _check(lib().moe_layer_nvfp4(ctypes.byref(shape), _ptr(logits), _ptr(ids_in), _ptr(w_in), _ptr(x), _ptr(w13),
                                 _ptr(w13_bscale), _ptr(w13_scale), _ptr(w2), _ptr(w2_bscale), _ptr(w2_scale),
                                 _ptr(residual), _ptr(out), _ptr(ws), _wsb(ws), _stream(stream)), "moe_layer_nvfp4")


def moe_dispatch_noalloc(shape, x, topk_ids, counts, offsets, dest, sorted_pair, x_perm, device_status=None,
                         stream=None):
    """moe_dispatch without a workspace (static scratch inside the library)."""
    _check(lib().moe_dispatch_noalloc(ctypes.byref(shape), _ptr(x), _ptr(topk_ids), _ptr(counts), _ptr(offsets),
                                      _ptr(dest), _ptr(sorted_pair), _ptr(x_perm), _ptr(device_status),
                                      _stream(stream)), "moe_dispatch_noalloc")


def moe_status_read(ws, stream=None) -> int:
    st = ctypes.c_int(0)
    _check(lib().moe_status_read(_ptr(ws), _stream(stream), ctypes.byref(st)), "moe_status_read")
    return st.value


def moe_workspace_set_wait(ws, lookback_wait_ns: int, count_tile_skip: int = 0, stream=None):
    """Test controls of the count kernel's bounded look-back wait."""
    _check(lib().moe_workspace_set_wait(_ptr(ws), _wsb(ws), int(lookback_wait_ns), int(count_tile_skip),
                                        _stream(stream)), "moe_workspace_set_wait")


def moe_timeout_site_read(ws, stream=None) -> int:
    site = ctypes.c_int32(0)
    _check(lib().moe_timeout_site_read(_ptr(ws), _stream(stream), ctypes.byref(site)), "moe_timeout_site_read")
    return site.value


# ---- training ---------------------------------------------------------------
_TYPES = {torch.bfloat16: MOE_TYPE_BF16, torch.float32: MOE_TYPE_F32}


def _type(t):
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError(f"bfloat16 or float32 tensor expected, got {t.dtype}") from None


def _norm_shape(x, gamma, *others):
    """(rows, hidden) of a layer norm over x's last dimension; the other tensors match it."""
    hidden = gamma.numel()
    if gamma.dim() != 1 or x.dim() < 1 or x.shape[-1] != hidden:
        raise ValueError(f"layer norm: weight of {tuple(gamma.shape)} for an input of {tuple(x.shape)}")
    for t in others:
        if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
            raise ValueError(f"layer norm: {tuple(t.shape)} {t.dtype} beside an input of {tuple(x.shape)} {x.dtype}")
    return x.numel() // hidden, hidden


def _stat(t, n, what):
    if t is not None and (t.dtype != torch.float32 or t.numel() != n):
        raise ValueError(f"layer norm: {what} must be float32 with {n} elements, got {t.dtype} {tuple(t.shape)}")
    return t


def moe_layernorm(x, gamma, beta, eps, y, mean=None, rstd=None, stream=None):
    """Layer norm over x's last dimension into y (and the rows' mean and rstd)."""
    rows, hidden = _norm_shape(x, gamma, y)
    if beta.shape != gamma.shape or beta.dtype != gamma.dtype:
        raise ValueError("layer norm: gamma and beta differ in shape or type")
    _check(lib().moe_layernorm(rows, hidden, _type(x), _type(gamma), _ptr(x), _ptr(gamma), _ptr(beta), float(eps),
                               _ptr(y), _ptr(_stat(mean, rows, "mean")), _ptr(_stat(rstd, rows, "rstd")),
                               _stream(stream)), "moe_layernorm")


def moe_layernorm_scratch_size(rows: int, hidden: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_layernorm_scratch_size(int(rows), int(hidden), ctypes.byref(n)), "moe_layernorm_scratch_size")
    return n.value


def layernorm_scratch(rows: int, hidden: int, device="cuda") -> torch.Tensor:
    """The scratch moe_layernorm_backward needs for this many rows."""
    return torch.empty(moe_layernorm_scratch_size(rows, hidden), dtype=torch.uint8, device=device)


def moe_layernorm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, scratch, dres=None, stream=None):
    """Gradient of moe_layernorm: dx (plus dres, the residual branch's gradient), dgamma, dbeta."""
    rows, hidden = _norm_shape(x, gamma, dy, dx, dres)
    _check(lib().moe_layernorm_backward(rows, hidden, _type(x), _type(gamma), _ptr(dy), _ptr(x), _ptr(gamma),
                                        _ptr(_stat(mean, rows, "mean")), _ptr(_stat(rstd, rows, "rstd")), _ptr(dres),
                                        _ptr(dx), _ptr(_stat(dgamma, hidden, "dgamma")),
                                        _ptr(_stat(dbeta, hidden, "dbeta")), _ptr(scratch), _wsb(scratch),
                                        _stream(stream)), "moe_layernorm_backward")


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _arg(t, dtype, n, what):
    """The address of a tensor with `n` elements of `dtype` at least (a kernel reads or
    writes that many); None and plain addresses pass as they are."""
    try:
        if t.dtype is dtype and t.numel() >= n and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        return _ptr(t)
    if t.dtype is not dtype or t.numel() < n:
        raise ValueError(f"{what}: {dtype} with {n} elements at least expected, got {t.dtype} {tuple(t.shape)}")
    return _ptr(t)


class _Counts(NamedTuple):
    """Elements of the training calls' tensors."""
    x: int          # [T, H]
    pairs: int      # [T, k]
    rows: int       # [T*k, H]
    logits: int     # [T, E]
    logits8: int    # [T, 8 * ceil(E / 8)]
    bounds: int     # [E + 1]
    pre: int        # [T*k, up]
    h: int          # [T*k, I]
    w_gate: int     # [E, H]
    w13: int        # [E, up, H]
    w2: int         # [E, H, I]


@functools.lru_cache(maxsize=256)
def _counts_of(fields: bytes) -> _Counts:
    s = moe_shape.from_buffer_copy(fields)
    T, H, E, I, R = s.tokens, s.hidden, s.experts, s.inter, s.tokens * s.top_k
    up = 2 * I if s.act == MOE_ACT_SWIGLU else I
    return _Counts(T * H, R, R * H, T * E, T * ((E + 7) // 8 * 8), E + 1, R * up, R * I, E * H, E * up * H, E * H * I)


def moe_combine_backward(shape, dout, y_perm, dest, topk_w, dy_perm, dtopk_w, ws, stream=None):
    """Gradient of moe_combine: dy_perm, and dtopk_w unless it is None."""
    n = _counts_of(bytes(shape))
    st = (_lib or lib()).moe_combine_backward(shape, _arg(dout, _BF16, n.x, "dout"),
                                              _arg(y_perm, _BF16, n.rows, "y_perm"),
                                              _arg(dest, _I32, n.pairs, "dest"),
                                              _arg(topk_w, _F32, n.pairs, "topk_w"),
                                              _arg(dy_perm, _BF16, n.rows, "dy_perm"),
                                              _arg(dtopk_w, _F32, n.pairs, "dtopk_w"), _ptr(ws), _wsb(ws),
                                              _stream(stream))
    if st:
        raise MoEError(st, "moe_combine_backward")


def moe_dispatch_backward(shape, dx_perm, dest, dx, ws, stream=None, add=None):
    """Gradient of moe_dispatch's row copy, plus `add`."""
    n = _counts_of(bytes(shape))
    st = (_lib or lib()).moe_dispatch_backward(shape, _arg(dx_perm, _BF16, n.rows, "dx_perm"),
                                               _arg(dest, _I32, n.pairs, "dest"), _arg(add, _BF16, n.x, "add"),
                                               _arg(dx, _BF16, n.x, "dx"), _ptr(ws), _wsb(ws), _stream(stream))
    if st:
        raise MoEError(st, "moe_dispatch_backward")


def moe_route_backward(shape, topk_ids, topk_w, dtopk_w, dlogits, ws, stream=None):
    n = _counts_of(bytes(shape))
    st = (_lib or lib()).moe_route_backward(shape, _arg(topk_ids, _I32, n.pairs, "topk_ids"),
                                            _arg(topk_w, _F32, n.pairs, "topk_w"),
                                            _arg(dtopk_w, _F32, n.pairs, "dtopk_w"),
                                            _arg(dlogits, _F32, n.logits, "dlogits"), _ptr(ws), _wsb(ws),
                                            _stream(stream))
    if st:
        raise MoEError(st, "moe_route_backward")


def moe_route_sigmoid_backward(shape, logits, topk_ids, route_scale, dtopk_w, dlogits, ws, stream=None):
    n = _counts_of(bytes(shape))
    st = (_lib or lib()).moe_route_sigmoid_backward(shape, _arg(logits, _F32, n.logits, "logits"),
                                                    _arg(topk_ids, _I32, n.pairs, "topk_ids"), float(route_scale),
                                                    _arg(dtopk_w, _F32, n.pairs, "dtopk_w"),
                                                    _arg(dlogits, _F32, n.logits, "dlogits"), _ptr(ws), _wsb(ws),
                                                    _stream(stream))
    if st:
        raise MoEError(st, "moe_route_sigmoid_backward")


def _wgrad(dw, add):
    """The moe_wgrad value of a weight gradient's tensor."""
    if dw is None:
        return MOE_WGRAD_BF16
    if dw.dtype is _F32:
        return MOE_WGRAD_F32_ADD if add else MOE_WGRAD_F32
    _type(dw)
    if add:
        raise ValueError("weight gradients are accumulated in float32")
    return MOE_WGRAD_BF16


def moe_gate_backward(shape, dlogits, x, w_gate, dlogits_bf16, dx, dw_gate, ws, stream=None, add=False):
    """dx (None: skipped) and dw_gate (None: skipped; bfloat16 or float32, `add` accumulates into
    float32) from dlogits, rounded into dlogits_bf16 [T, 8 * ceil(E / 8)] on the way."""
    n, mode = _counts_of(bytes(shape)), _wgrad(dw_gate, add)
    st = (_lib or lib()).moe_gate_backward(shape, _arg(dlogits, _F32, n.logits, "dlogits"), _arg(x, _BF16, n.x, "x"),
                                           _arg(w_gate, _BF16, n.w_gate, "w_gate"),
                                           _arg(dlogits_bf16, _BF16, n.logits8, "dlogits_bf16"),
                                           _arg(dx, _BF16, n.x, "dx"),
                                           _arg(dw_gate, _F32 if mode else _BF16, n.w_gate, "dw_gate"), mode,
                                           _ptr(ws), _wsb(ws), _stream(stream))
    if st:
        raise MoEError(st, "moe_gate_backward")


def moe_expert_up_train(shape, x_perm, offsets, w13, pre, h, ws, stream=None):
    """Up projection that also keeps its pre-activations for the backward pass."""
    n = _counts_of(bytes(shape))
    st = (_lib or lib()).moe_expert_up_train(shape, _arg(x_perm, _BF16, n.rows, "x_perm"),
                                             _arg(offsets, _I32, n.bounds, "offsets"), _arg(w13, _BF16, n.w13, "w13"),
                                             _arg(pre, _BF16, n.pre, "pre"), _arg(h, _BF16, n.h, "h"), _ptr(ws),
                                             _wsb(ws), _stream(stream))
    if st:
        raise MoEError(st, "moe_expert_up_train")


def moe_expert_down_backward(shape, dy_perm, offsets, w2, pre, h, dpre, dw2, ws, stream=None, add=False):
    """dpre (None: skipped) and dw2 (None: skipped; bfloat16 or float32, `add` accumulates into float32)."""
    n, mode = _counts_of(bytes(shape)), _wgrad(dw2, add)
    st = (_lib or lib()).moe_expert_down_backward(shape, _arg(dy_perm, _BF16, n.rows, "dy_perm"),
                                                  _arg(offsets, _I32, n.bounds, "offsets"),
                                                  _arg(w2, _BF16, n.w2, "w2"), _arg(pre, _BF16, n.pre, "pre"),
                                                  _arg(h, _BF16, n.h, "h"), _arg(dpre, _BF16, n.pre, "dpre"),
                                                  _arg(dw2, _F32 if mode else _BF16, n.w2, "dw2"), mode, _ptr(ws),
                                                  _wsb(ws), _stream(stream))
    if st:
        raise MoEError(st, "moe_expert_down_backward")


def moe_expert_up_backward(shape, dpre, offsets, x_perm, w13, dx_perm, dw13, ws, stream=None, add=False):
    """dx_perm (None: skipped) and dw13 (None: skipped; types as dw2)."""
    n, mode = _counts_of(bytes(shape)), _wgrad(dw13, add)
    st = (_lib or lib()).moe_expert_up_backward(shape, _arg(dpre, _BF16, n.pre, "dpre"),
                                                _arg(offsets, _I32, n.bounds, "offsets"),
                                                _arg(x_perm, _BF16, n.rows, "x_perm"), _arg(w13, _BF16, n.w13, "w13"),
                                                _arg(dx_perm, _BF16, n.rows, "dx_perm"),
                                                _arg(dw13, _F32 if mode else _BF16, n.w13, "dw13"), mode, _ptr(ws),
                                                _wsb(ws), _stream(stream))
    if st:
        raise MoEError(st, "moe_expert_up_backward")


def moe_ep_plan(experts: int, world: int, rank: int, capacity: int, counts_all):
    """Host-side plan of the expert-parallel exchange (numpy in, numpy out):
    -> (status, dict(send_offsets [E+1], recv_offsets [el+1], recv_slot [world, el],
    peer_send [world], peer_recv [world])).  The status is MOE_OK or
    MOE_ERR_CAPACITY (the plan is written either way); other errors raise."""
    import numpy as np
    ca = np.ascontiguousarray(counts_all, dtype=np.int32)
    if ca.shape != (world, experts):
        raise ValueError(f"counts_all must be [{world}, {experts}], got {ca.shape}")
    e0, e1 = rank * experts // world, (rank + 1) * experts // world
    out = dict(send_offsets=np.zeros(experts + 1, np.int32), recv_offsets=np.zeros(e1 - e0 + 1, np.int32),
               recv_slot=np.zeros((world, e1 - e0), np.int32), peer_send=np.zeros(world, np.int32),
               peer_recv=np.zeros(world, np.int32))
    p = lambda a: ctypes.c_void_p(a.ctypes.data)
    st = lib().moe_ep_plan(experts, world, rank, capacity, p(ca), p(out["send_offsets"]), p(out["recv_offsets"]),
                           p(out["recv_slot"]), p(out["peer_send"]), p(out["peer_recv"]))
    if st not in (MOE_OK, MOE_ERR_CAPACITY):
        raise MoEError(st, "moe_ep_plan")
    return st, out
