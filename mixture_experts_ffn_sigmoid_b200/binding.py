"""ctypes binding of ``libmoe_b200.so`` (declared in ``include/moe.h``).

Argument marshalling only: every function here checks that each torch
tensor has the dtype the entry point expects and at least as many elements as
the library will read or write through it (a short buffer would be an
out-of-bounds access on the GPU), that it is a contiguous CUDA tensor, passes
the device pointers and the current CUDA stream to the C entry point of the
same name, and raises ``MoEError`` on a non-OK status. All compute runs in the library's CUDA kernels; there is no other
path. If the library is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import os
from typing import Optional

import torch

from .inputs import MoEConfig, NormConfig, OrthoConfig

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_MISALIGNED = 2
MOE_ERR_UNSUPPORTED = 3
MOE_ERR_WORKSPACE_TOO_SMALL = 4
MOE_ERR_CUDA = 5
MOE_ERR_TIMEOUT = 6

MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1

EXPORTED = ("moe_check_config", "moe_workspace_size", "moe_route", "moe_permute",
            "moe_expert_swiglu", "moe_expert_gate_up", "moe_expert_gate_up_gather", "moe_expert_down",
            "moe_combine", "moe_forward", "moe_get_device_error",
            "moe_selftest_wait_timeout", "moe_route_noalloc", "moe_route_noalloc_device_error",
            "moe_forward_gathers_rows", "moe_route_maps", "moe_route_maps_supported",
            "moe_balance_update",
            "moe_expert_gelu", "moe_forward_gelu", "moe_backward_workspace_size", "moe_backward",
            "moe_forward_train", "moe_backward_saved", "moe_w4_quantize", "moe_w4_dequantize",
            "moe_expert_swiglu_w4", "moe_forward_w4", "moe_ortho_workspace_size", "moe_orthogonalize", "moe_muon_step",
            "moe_residual_norm",
            "moe_residual_norm_backward_workspace_size", "moe_residual_norm_backward", "moe_status_string")


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class CConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("f", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate_mode", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("route_scale", ctypes.c_float),
                ("f_shared", ctypes.c_int32)]


class CW4Matrix(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p)]


class COrthoConfig(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("steps", ctypes.c_int32), ("eps", ctypes.c_float)]


class CNormConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate_tokens", ctypes.c_int32), ("eps", ctypes.c_float), ("alpha", ctypes.c_float),
                ("beta", ctypes.c_float), ("w_offset", ctypes.c_float)]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Load the CUDA library once; raise if it is not there."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m mixture_experts_ffn_sigmoid_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        vp, sz, i32p, f32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p
        cfgp, ncfgp = ctypes.POINTER(CConfig), ctypes.POINTER(CNormConfig)
        w4p, ocfgp = ctypes.POINTER(CW4Matrix), ctypes.POINTER(COrthoConfig)
        i32, i64, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        sig = {
            "moe_check_config": (ctypes.c_int, [cfgp]),
            "moe_workspace_size": (sz, [cfgp]),
            "moe_route": (ctypes.c_int, [cfgp, vp, vp, f32p, i32p, f32p, i32p, i32p, vp, sz, vp]),
            "moe_permute": (ctypes.c_int, [cfgp, vp, i32p, i32p, vp, i32p, i32p, vp, sz, vp]),
            "moe_expert_swiglu": (ctypes.c_int, [cfgp, vp, i32p, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                 vp, sz, vp]),
            "moe_expert_gate_up": (ctypes.c_int, [cfgp, vp, i32p, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_expert_gate_up_gather": (ctypes.c_int, [cfgp, vp, i32p, i32p, vp, vp, vp, vp, vp, vp, vp,
                                                         sz, vp]),
            "moe_expert_down": (ctypes.c_int, [cfgp, vp, i32p, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_combine": (ctypes.c_int, [cfgp, vp, i32p, f32p, vp, vp, vp]),
            "moe_forward": (ctypes.c_int, [cfgp, vp, vp, f32p, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_get_device_error": (ctypes.c_int, [vp, vp]),
            "moe_selftest_wait_timeout": (ctypes.c_int, [vp, sz, ctypes.c_int64, vp]),
            "moe_route_noalloc": (ctypes.c_int, [cfgp, vp, vp, f32p, i32p, f32p, i32p, i32p, vp]),
            "moe_route_noalloc_device_error": (ctypes.c_int, [vp]),
            "moe_forward_gathers_rows": (ctypes.c_int, [cfgp, vp]),
            "moe_route_maps": (ctypes.c_int, [cfgp, vp, vp, f32p, i32p, f32p, i32p, i32p, i32p, i32p, vp, sz, vp]),
            "moe_route_maps_supported": (ctypes.c_int, [cfgp]),
            "moe_balance_update": (ctypes.c_int, [cfgp, i32p, f32p, ctypes.c_float, f32p, vp]),
            "moe_expert_gelu": (ctypes.c_int, [cfgp, vp, i32p, vp, f32p, vp, f32p, vp, vp, sz, vp]),
            "moe_forward_gelu": (ctypes.c_int, [cfgp, vp, vp, f32p, vp, f32p, vp, f32p, vp, vp, sz, vp]),
            "moe_backward_workspace_size": (sz, [cfgp]),
            "moe_forward_train": (ctypes.c_int, [cfgp, vp, vp, f32p, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_backward_saved": (ctypes.c_int, [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                  vp, vp, vp, vp, sz, vp]),
            "moe_backward": (ctypes.c_int, [cfgp, vp, vp, f32p, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                            vp, vp, vp, vp, sz, vp]),
            "moe_ortho_workspace_size": (sz, [ocfgp]),
            "moe_orthogonalize": (ctypes.c_int, [ocfgp, vp, vp, vp, vp, sz, vp]),
            "moe_muon_step": (ctypes.c_int, [ocfgp, vp, vp, vp, vp, i32, f32, f32, i32, f32, f32, vp, sz, vp]),
            "moe_w4_quantize": (ctypes.c_int, [i64, i32, i32, i32, vp, w4p, vp]),
            "moe_w4_dequantize": (ctypes.c_int, [i64, i32, i32, i32, w4p, vp, vp]),
            "moe_expert_swiglu_w4": (ctypes.c_int, [cfgp, i32, vp, i32p, i32p, w4p, w4p, w4p, vp, w4p, w4p, w4p, vp,
                                                    vp, vp, sz, vp]),
            "moe_forward_w4": (ctypes.c_int, [cfgp, i32, vp, vp, f32p, w4p, w4p, w4p, w4p, w4p, w4p, vp, vp, sz, vp]),
            "moe_residual_norm": (ctypes.c_int, [ncfgp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "moe_residual_norm_backward_workspace_size": (sz, [ncfgp]),
            "moe_residual_norm_backward": (ctypes.c_int, [ncfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                          sz, vp]),
            "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def make_config(cfg: MoEConfig, T: Optional[int] = None) -> CConfig:
    return CConfig(T=cfg.T if T is None else T, d=cfg.d, E=cfg.E, k=cfg.k, f=cfg.f,
                   dtype=MOE_DTYPE_F32 if cfg.dtype == "f32" else MOE_DTYPE_BF16,
                   gate_mode=cfg.gate_mode, n_groups=cfg.n_groups, topk_groups=cfg.topk_groups,
                   route_scale=cfg.route_scale, f_shared=cfg.f_shared)


def _cfg(c) -> CConfig:
    return c if isinstance(c, CConfig) else make_config(c)


_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


def _dt(c: CConfig) -> torch.dtype:
    return torch.float32 if c.dtype == MOE_DTYPE_F32 else torch.bfloat16


def _need(t, name: str, numel: int, dtype: torch.dtype, required: bool = True):
    """Refuse a tensor the library would overrun or misread: wrong dtype, or
    fewer than ``numel`` elements. None passes where the C entry point takes
    NULL (``required=False``) and where it reads or writes nothing through the
    pointer (``numel == 0``, e.g. token arrays when T = 0)."""
    if t is None:
        if required and numel > 0:
            raise ValueError(f"{name} is required")
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, not {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, needs at least {numel}")


def _need_routing_io(c: CConfig, x, w_router, bias, topk_idx, topk_gate, expert_counts, expert_offsets):
    T, d, E, k, dt = c.T, c.d, c.E, c.k, _dt(c)
    _need(x, "x", T * d, dt)
    _need(w_router, "w_router", E * d, dt)
    _need(bias, "bias", E, _F32, required=False)
    _need(topk_idx, "topk_idx", T * k, _I32)
    _need(topk_gate, "topk_gate", T * k, _F32)
    _need(expert_counts, "expert_counts", E, _I32)
    _need(expert_offsets, "expert_offsets", E + 1, _I32)


def _need_weights(c: CConfig, w1, w3, w2, ws1, ws3, ws2, prefix: str = ""):
    d, E, f, fs, dt = c.d, c.E, c.f, c.f_shared, _dt(c)
    sh = fs > 0
    _need(w1, prefix + "w1", E * f * d, dt)
    _need(w3, prefix + "w3", E * f * d, dt)
    _need(w2, prefix + "w2", E * d * f, dt)
    _need(ws1, prefix + "ws1", fs * d, dt, required=sh)
    _need(ws3, prefix + "ws3", fs * d, dt, required=sh)
    _need(ws2, prefix + "ws2", d * fs, dt, required=sh)


def _need_ws(workspace):
    if workspace is None:
        raise ValueError("workspace is required")
    _need(workspace, "workspace", 0, _U8)


def _need_block(c: CConfig, x, w_router, bias, w1, w3, w2, ws1, ws3, ws2, y, workspace):
    """Inputs of the whole block (y checked unless None is passed for it)."""
    dt = _dt(c)
    _need(x, "x", c.T * c.d, dt)
    _need(w_router, "w_router", c.E * c.d, dt)
    _need(bias, "bias", c.E, _F32, required=False)
    _need_weights(c, w1, w3, w2, ws1, ws3, ws2)
    if y is not None:
        _need(y, "y", c.T * c.d, dt)
    _need_ws(workspace)


def _need_grads(c: CConfig, dy, dx, dw_router, dw1, dw3, dw2, dws1, dws3, dws2):
    dt = _dt(c)
    _need(dy, "dy", c.T * c.d, dt)
    _need(dx, "dx", c.T * c.d, dt)
    _need(dw_router, "dw_router", c.E * c.d, dt)
    _need_weights(c, dw1, dw3, dw2, dws1, dws3, dws2, prefix="d")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptrs(*tensors):
    """Device addresses (None for None) of contiguous CUDA tensors, all on the
    current device: kernels are launched there, and another GPU's memory may
    not be reachable from it."""
    dev = None
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if not t.is_cuda:
            raise ValueError("tensor must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        if dev is None:
            dev = torch.cuda.current_device()
        if t.get_device() != dev:
            raise ValueError(f"tensor lives on cuda:{t.get_device()}, the current device is cuda:{dev}")
        out.append(t.data_ptr())
    return out


_Tensor = torch.Tensor


def _args(*specs):
    """Addresses of (tensor, name, least elements, dtype, required) in order.
    One pass over tensors that are as they should be (a decode step makes many
    small calls); anything else goes through _need and _ptrs for its error."""
    dev = None
    out = []
    for t, _, n, dt, required in specs:
        if t is None:
            if required and n > 0:
                break
            out.append(None)
        elif isinstance(t, _Tensor) and t.dtype is dt and t.numel() >= n and t.is_contiguous():
            on = t.get_device()
            if on != dev:                  # the first: on the current device (below 0: on the host)
                if dev is not None or on < 0 or on != torch._C._cuda_getDevice():
                    break
                dev = on
            out.append(t.data_ptr())
        else:
            break
    else:
        return out
    for t, name, n, dt, required in specs:
        if name == "workspace":
            _need_ws(t)
        else:
            _need(t, name, n, dt, required)
    return _ptrs(*(spec[0] for spec in specs))


def _raw_stream(stream):
    """The stream's handle; the current device's current stream for None."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _allocating_on(stream):
    """Context in which torch allocates memory of ``stream`` (None: the current
    stream, a Stream or a raw handle). The allocator hands a tensor's memory on
    in the order of the stream it was allocated on, so what kernels on another
    one write or read could still be, or already be again, someone else's."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_raw_stream(stream))
    return torch.cuda.stream(stream)


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where)


def check_config(cfg) -> int:
    return lib().moe_check_config(ctypes.byref(_cfg(cfg)))


def workspace_size(cfg) -> int:
    return lib().moe_workspace_size(ctypes.byref(_cfg(cfg)))


def alloc_workspace(cfg, device="cuda") -> torch.Tensor:
    n = workspace_size(cfg)
    if n == 0:
        raise MoEError(check_config(cfg) or MOE_ERR_INVALID_ARG, "moe_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_route(cfg, x, w_router, bias, topk_idx, topk_gate, expert_counts, expert_offsets,
              workspace, stream=None):
    c = _cfg(cfg)
    _need_routing_io(c, x, w_router, bias, topk_idx, topk_gate, expert_counts, expert_offsets)
    _need_ws(workspace)
    _check(lib().moe_route(ctypes.byref(c), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(topk_idx),
                           _ptr(topk_gate), _ptr(expert_counts), _ptr(expert_offsets),
                           _ptr(workspace), workspace.numel(), _stream(stream)), "moe_route")


def moe_route_maps(cfg, x, w_router, bias, topk_idx, topk_gate, expert_counts, expert_offsets, perm_src,
                   inv_row, workspace, stream=None):
    """moe_route plus the maps-only permute in one launch (one-tile batches)."""
    c = _cfg(cfg)
    _need_routing_io(c, x, w_router, bias, topk_idx, topk_gate, expert_counts, expert_offsets)
    _need(perm_src, "perm_src", c.T * c.k, _I32)
    _need(inv_row, "inv_row", c.T * c.k, _I32)
    _need_ws(workspace)
    _check(lib().moe_route_maps(ctypes.byref(c), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(topk_idx),
                                _ptr(topk_gate), _ptr(expert_counts), _ptr(expert_offsets), _ptr(perm_src),
                                _ptr(inv_row), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_route_maps")


def moe_route_maps_supported(cfg) -> bool:
    """Whether moe_route_maps runs for cfg (else it returns MOE_ERR_UNSUPPORTED)."""
    r = lib().moe_route_maps_supported(ctypes.byref(_cfg(cfg)))
    if r < 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_route_maps_supported")
    return r == 1


def moe_permute(cfg, x, topk_idx, expert_offsets, x_perm, perm_src, inv_row, workspace, stream=None):
    c = _cfg(cfg)
    R, dt = c.T * c.k, _dt(c)
    _need(x, "x", c.T * c.d, dt, required=x_perm is not None)
    _need(topk_idx, "topk_idx", R, _I32)
    _need(expert_offsets, "expert_offsets", c.E + 1, _I32)
    _need(x_perm, "x_perm", R * c.d, dt, required=False)
    _need(perm_src, "perm_src", R, _I32)
    _need(inv_row, "inv_row", R, _I32)
    _need_ws(workspace)
    _check(lib().moe_permute(ctypes.byref(c), _ptr(x), _ptr(topk_idx), _ptr(expert_offsets),
                             _ptr(x_perm), _ptr(perm_src), _ptr(inv_row), _ptr(workspace),
                             workspace.numel(), _stream(stream)), "moe_permute")


def moe_expert_swiglu(cfg, x_perm, expert_offsets, w1, w3, w2, x_shared, ws1, ws3, ws2, y_perm,
                      y_shared, workspace, stream=None):
    c = _cfg(cfg)
    R, dt, sh = c.T * c.k, _dt(c), c.f_shared > 0
    _need(x_perm, "x_perm", R * c.d, dt)
    _need(expert_offsets, "expert_offsets", c.E + 1, _I32)
    _need_weights(c, w1, w3, w2, ws1, ws3, ws2)
    _need(x_shared, "x_shared", c.T * c.d, dt, required=sh)
    _need(y_perm, "y_perm", R * c.d, dt)
    _need(y_shared, "y_shared", c.T * c.d, dt, required=sh)
    _need_ws(workspace)
    _check(lib().moe_expert_swiglu(ctypes.byref(c), _ptr(x_perm), _ptr(expert_offsets), _ptr(w1),
                                   _ptr(w3), _ptr(w2), _ptr(x_shared), _ptr(ws1), _ptr(ws3),
                                   _ptr(ws2), _ptr(y_perm), _ptr(y_shared), _ptr(workspace),
                                   workspace.numel(), _stream(stream)), "moe_expert_swiglu")


def moe_expert_gate_up(cfg, x_perm, expert_offsets, w1, w3, x_shared, ws1, ws3, h, h_shared,
                       workspace, stream=None):
    c = _cfg(cfg)
    R, dt, sh, fs = c.T * c.k, _dt(c), c.f_shared > 0, c.f_shared
    _need(x_perm, "x_perm", R * c.d, dt)
    _need(expert_offsets, "expert_offsets", c.E + 1, _I32)
    _need(w1, "w1", c.E * c.f * c.d, dt)
    _need(w3, "w3", c.E * c.f * c.d, dt)
    _need(x_shared, "x_shared", c.T * c.d, dt, required=sh)
    _need(ws1, "ws1", fs * c.d, dt, required=sh)
    _need(ws3, "ws3", fs * c.d, dt, required=sh)
    _need(h, "h", R * c.f, dt)
    _need(h_shared, "h_shared", c.T * fs, dt, required=sh)
    _need_ws(workspace)
    _check(lib().moe_expert_gate_up(ctypes.byref(c), _ptr(x_perm), _ptr(expert_offsets), _ptr(w1),
                                    _ptr(w3), _ptr(x_shared), _ptr(ws1), _ptr(ws3), _ptr(h),
                                    _ptr(h_shared), _ptr(workspace), workspace.numel(),
                                    _stream(stream)), "moe_expert_gate_up")


def moe_expert_gate_up_gather(cfg, x, perm_src, expert_offsets, w1, w3, ws1, ws3, h, h_shared,
                              workspace, stream=None):
    c = _cfg(cfg)
    R, dt, sh, fs = c.T * c.k, _dt(c), c.f_shared > 0, c.f_shared
    _need(x, "x", c.T * c.d, dt)
    _need(perm_src, "perm_src", R, _I32)
    _need(expert_offsets, "expert_offsets", c.E + 1, _I32)
    _need(w1, "w1", c.E * c.f * c.d, dt)
    _need(w3, "w3", c.E * c.f * c.d, dt)
    _need(ws1, "ws1", fs * c.d, dt, required=sh)
    _need(ws3, "ws3", fs * c.d, dt, required=sh)
    _need(h, "h", R * c.f, dt)
    _need(h_shared, "h_shared", c.T * fs, dt, required=sh)
    _need_ws(workspace)
    _check(lib().moe_expert_gate_up_gather(ctypes.byref(c), _ptr(x), _ptr(perm_src), _ptr(expert_offsets),
                                           _ptr(w1), _ptr(w3), _ptr(ws1), _ptr(ws3), _ptr(h),
                                           _ptr(h_shared), _ptr(workspace), workspace.numel(),
                                           _stream(stream)), "moe_expert_gate_up_gather")


def moe_expert_down(cfg, h, expert_offsets, w2, h_shared, ws2, y_perm, y_shared, workspace,
                    stream=None):
    c = _cfg(cfg)
    R, dt, sh, fs = c.T * c.k, _dt(c), c.f_shared > 0, c.f_shared
    _need(h, "h", R * c.f, dt)
    _need(expert_offsets, "expert_offsets", c.E + 1, _I32)
    _need(w2, "w2", c.E * c.d * c.f, dt)
    _need(h_shared, "h_shared", c.T * fs, dt, required=sh)
    _need(ws2, "ws2", c.d * fs, dt, required=sh)
    _need(y_perm, "y_perm", R * c.d, dt)
    _need(y_shared, "y_shared", c.T * c.d, dt, required=sh)
    _need_ws(workspace)
    _check(lib().moe_expert_down(ctypes.byref(c), _ptr(h), _ptr(expert_offsets), _ptr(w2),
                                 _ptr(h_shared), _ptr(ws2), _ptr(y_perm), _ptr(y_shared),
                                 _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_expert_down")


def moe_combine(cfg, y_perm, inv_row, topk_gate, y_shared, y, stream=None):
    c = _cfg(cfg)
    R, dt = c.T * c.k, _dt(c)
    _need(y_perm, "y_perm", R * c.d, dt)
    _need(inv_row, "inv_row", R, _I32)
    _need(topk_gate, "topk_gate", R, _F32)
    _need(y_shared, "y_shared", c.T * c.d, dt, required=False)
    _need(y, "y", c.T * c.d, dt)
    _check(lib().moe_combine(ctypes.byref(c), _ptr(y_perm), _ptr(inv_row), _ptr(topk_gate),
                             _ptr(y_shared), _ptr(y), _stream(stream)), "moe_combine")


def moe_forward(cfg, x, w_router, bias, w1, w3, w2, ws1, ws3, ws2, y, workspace, stream=None):
    c = _cfg(cfg)
    _need_block(c, x, w_router, bias, w1, w3, w2, ws1, ws3, ws2, y, workspace)
    _check(lib().moe_forward(ctypes.byref(c), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w1),
                             _ptr(w3), _ptr(w2), _ptr(ws1), _ptr(ws3), _ptr(ws2), _ptr(y),
                             _ptr(workspace), workspace.numel(), _stream(stream)), "moe_forward")


def moe_expert_gelu(cfg, x_perm, expert_offsets, w1, b1, w2, b2, y_perm, workspace, stream=None):
    """Generic experts on packed rows: y = W2 GELU(W1 x + b1) + b2 per segment."""
    c = _cfg(cfg)
    R, dt = c.T * c.k, _dt(c)
    _need(x_perm, "x_perm", R * c.d, dt)
    _need(expert_offsets, "expert_offsets", c.E + 1, _I32)
    _need(w1, "w1", c.E * c.f * c.d, dt)
    _need(b1, "b1", c.E * c.f, _F32, required=False)
    _need(w2, "w2", c.E * c.d * c.f, dt)
    _need(b2, "b2", c.E * c.d, _F32, required=False)
    _need(y_perm, "y_perm", R * c.d, dt)
    _need_ws(workspace)
    _check(lib().moe_expert_gelu(ctypes.byref(c), _ptr(x_perm), _ptr(expert_offsets), _ptr(w1), _ptr(b1),
                                 _ptr(w2), _ptr(b2), _ptr(y_perm), _ptr(workspace), workspace.numel(),
                                 _stream(stream)), "moe_expert_gelu")


def moe_forward_gelu(cfg, x, w_router, bias, w1, b1, w2, b2, y, workspace, stream=None):
    """The block with generic GELU experts (no shared expert)."""
    c = _cfg(cfg)
    dt = _dt(c)
    _need(x, "x", c.T * c.d, dt)
    _need(w_router, "w_router", c.E * c.d, dt)
    _need(bias, "bias", c.E, _F32, required=False)
    _need(w1, "w1", c.E * c.f * c.d, dt)
    _need(b1, "b1", c.E * c.f, _F32, required=False)
    _need(w2, "w2", c.E * c.d * c.f, dt)
    _need(b2, "b2", c.E * c.d, _F32, required=False)
    _need(y, "y", c.T * c.d, dt)
    _need_ws(workspace)
    _check(lib().moe_forward_gelu(ctypes.byref(c), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w1),
                                  _ptr(b1), _ptr(w2), _ptr(b2), _ptr(y), _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "moe_forward_gelu")


def backward_workspace_size(cfg) -> int:
    c = _cfg(cfg)
    return int(lib().moe_backward_workspace_size(ctypes.byref(c)))


def alloc_backward_workspace(cfg, device="cuda") -> torch.Tensor:
    n = backward_workspace_size(cfg)
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_backward_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_backward(cfg, x, w_router, bias, w1, w3, w2, ws1, ws3, ws2, dy, dx, dw_router, dw1, dw3, dw2,
                 dws1, dws3, dws2, workspace, stream=None):
    """Gradients of the block with respect to x and every weight, given dy."""
    c = _cfg(cfg)
    _need_block(c, x, w_router, bias, w1, w3, w2, ws1, ws3, ws2, None, workspace)
    _need_grads(c, dy, dx, dw_router, dw1, dw3, dw2, dws1, dws3, dws2)
    _check(lib().moe_backward(ctypes.byref(c), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w1), _ptr(w3),
                              _ptr(w2), _ptr(ws1), _ptr(ws3), _ptr(ws2), _ptr(dy), _ptr(dx), _ptr(dw_router),
                              _ptr(dw1), _ptr(dw3), _ptr(dw2), _ptr(dws1), _ptr(dws3), _ptr(dws2),
                              _ptr(workspace), workspace.numel(), _stream(stream)), "moe_backward")


def moe_forward_train(cfg, x, w_router, bias, w1, w3, w2, ws1, ws3, ws2, y, workspace, stream=None):
    """moe_forward that keeps routing and pre-activations in a backward-size workspace."""
    c = _cfg(cfg)
    _need_block(c, x, w_router, bias, w1, w3, w2, ws1, ws3, ws2, y, workspace)
    _check(lib().moe_forward_train(ctypes.byref(c), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w1), _ptr(w3),
                                   _ptr(w2), _ptr(ws1), _ptr(ws3), _ptr(ws2), _ptr(y), _ptr(workspace),
                                   workspace.numel(), _stream(stream)), "moe_forward_train")


def moe_backward_saved(cfg, x, w_router, w1, w3, w2, ws1, ws3, ws2, dy, dx, dw_router, dw1, dw3, dw2,
                       dws1, dws3, dws2, workspace, stream=None):
    """moe_backward on the state moe_forward_train left in `workspace`."""
    c = _cfg(cfg)
    _need_block(c, x, w_router, None, w1, w3, w2, ws1, ws3, ws2, None, workspace)
    _need_grads(c, dy, dx, dw_router, dw1, dw3, dw2, dws1, dws3, dws2)
    _check(lib().moe_backward_saved(ctypes.byref(c), _ptr(x), _ptr(w_router), _ptr(w1), _ptr(w3), _ptr(w2),
                                    _ptr(ws1), _ptr(ws3), _ptr(ws2), _ptr(dy), _ptr(dx), _ptr(dw_router),
                                    _ptr(dw1), _ptr(dw3), _ptr(dw2), _ptr(dws1), _ptr(dws3), _ptr(dws2),
                                    _ptr(workspace), workspace.numel(), _stream(stream)), "moe_backward_saved")


def moe_route_noalloc(cfg, x, w_router, bias, topk_idx, topk_gate, expert_counts, expert_offsets,
                      stream=None):
    """moe_route with the router's scratch in the library's fixed device array."""
    c = _cfg(cfg)
    _need_routing_io(c, x, w_router, bias, topk_idx, topk_gate, expert_counts, expert_offsets)
    _check(lib().moe_route_noalloc(ctypes.byref(c), _ptr(x), _ptr(w_router), _ptr(bias),
                                   _ptr(topk_idx), _ptr(topk_gate), _ptr(expert_counts),
                                   _ptr(expert_offsets), _stream(stream)), "moe_route_noalloc")


def moe_route_noalloc_device_error(stream=None) -> int:
    """Status of moe_route_noalloc's bounded device waits on the current
    device (synchronises the stream, then reads and clears the fixed array's
    error word): MOE_OK or MOE_ERR_TIMEOUT."""
    return lib().moe_route_noalloc_device_error(_stream(stream))


def moe_forward_gathers_rows(cfg, x) -> bool:
    """Whether moe_forward's gate/up GEMM gathers the token rows of x itself
    (the permute then writes the maps only) rather than reading a packed copy."""
    r = lib().moe_forward_gathers_rows(ctypes.byref(_cfg(cfg)), _ptr(x))
    if r < 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_forward_gathers_rows")
    return r == 1


def moe_balance_update(cfg, expert_counts, bias, gamma: float, entropy=None, stream=None):
    """Aux-loss-free bias step in place on `bias` and/or the routing entropy."""
    c = _cfg(cfg)
    _need(expert_counts, "expert_counts", c.E, _I32)
    _need(bias, "bias", c.E, _F32, required=False)
    _need(entropy, "entropy", 1, _F32, required=False)
    _check(lib().moe_balance_update(ctypes.byref(c), _ptr(expert_counts), _ptr(bias), float(gamma),
                                    _ptr(entropy), _stream(stream)), "moe_balance_update")


# ------------------------------------------------------------- 4-bit weights
class W4Matrix:
    """A weight matrix (or stack of them) [..., K] in 4 bits with group scales:
    ``q`` uint8 [..., K/2] (even k in the low four bits), ``scale`` bf16
    [..., K/group], ``zero`` uint8 [..., K/group] or None for 8 everywhere.
    ``W = scale * (code - zero)``. The three tensors are the matrix's for its
    lifetime; their contents may change."""

    q = property(lambda self: self._tensors[0])
    scale = property(lambda self: self._tensors[1])
    zero = property(lambda self: self._tensors[2])

    def __init__(self, q, scale, zero=None, group: int = 128):
        _need(q, "q", 0, _U8)
        _need(scale, "scale", 0, torch.bfloat16)
        _need(zero, "zero", 0, _U8, required=False)
        if group not in (32, 64, 128):
            raise ValueError(f"group {group}: expected 32, 64 or 128")
        if q.dim() < 1 or (2 * q.shape[-1]) % group:
            raise ValueError(f"q: rows of {2 * q.shape[-1] if q.dim() else 0} codes are not whole groups of {group}")
        self._tensors, self.group = (q, scale, zero), group
        self.K = 2 * q.shape[-1]
        self.rows = q.numel() // q.shape[-1] if q.numel() else 0
        self._struct = self._ref = self._at = None
        for t, name in ((scale, "scale"), (zero, "zero")):
            if t is not None and t.numel() != self.rows * (self.K // group):
                raise ValueError(f"{name}: {t.numel()} elements, expected {self.rows * (self.K // group)}")

    @classmethod
    def empty(cls, *shape, group: int = 128, zero_points: bool = False, device="cuda") -> "W4Matrix":
        """Uninitialised buffers for a matrix (stack) of the given dense shape."""
        *lead, K = shape
        if group not in (32, 64, 128) or K % group:
            raise ValueError(f"rows of {K} are not whole groups of {group}")
        return cls(torch.empty(*lead, K // 2, dtype=_U8, device=device),
                   torch.empty(*lead, K // group, dtype=torch.bfloat16, device=device),
                   torch.empty(*lead, K // group, dtype=_U8, device=device) if zero_points else None, group)

    @classmethod
    def quantize(cls, w: torch.Tensor, group: int = 128, zero_points: bool = False, stream=None) -> "W4Matrix":
        """The 4-bit form of a dense bf16 or fp32 matrix (stack), in memory of ``stream``."""
        with _allocating_on(stream):
            m = cls.empty(*w.shape, group=group, zero_points=zero_points, device=w.device)
        moe_w4_quantize(w, m, stream)
        return m

    def _c(self):
        """Reference to the C struct. The matrix's own tensors are checked when it
        is first used, and again if one's storage has moved (``tensor.data = ``)
        or the current device is another."""
        q, scale, zero = self._tensors
        at = self._at
        if at is None or at != (q.data_ptr(), scale.data_ptr(), None if zero is None else zero.data_ptr(),
                                torch._C._cuda_getDevice()):
            groups = self.rows * (self.K // self.group)
            a = _args((q, "q", self.rows * (self.K // 2), _U8, True), (scale, "scale", groups, torch.bfloat16, True),
                      (zero, "zero", groups, _U8, False))
            self._struct = CW4Matrix(*a)
            self._ref, self._at = ctypes.byref(self._struct), (*a, torch._C._cuda_getDevice())
        return self._ref


def _dense_code(w, name: str) -> int:
    _need_tensor(w, name)
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name}: dtype {w.dtype}, expected float32 or bfloat16")
    return MOE_DTYPE_F32 if w.dtype == torch.float32 else MOE_DTYPE_BF16


def _need_tensor(t, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, not {type(t).__name__}")


def moe_w4_quantize(w, out: W4Matrix, stream=None):
    """Write the 4-bit form of the dense matrix w into out (zero points if it has room for them)."""
    code = _dense_code(w, "w")
    if w.numel() != out.rows * out.K:
        raise ValueError(f"w: {w.numel()} elements, out holds {out.rows * out.K}")
    (pw,) = _args((w, "w", 0, w.dtype, True))
    _check(lib().moe_w4_quantize(out.rows, out.K, code, out.group, pw, out._c(), _raw_stream(stream)),
           "moe_w4_quantize")


def moe_w4_dequantize(m: W4Matrix, w, stream=None):
    """Write the dense values of m into w (bf16 or fp32)."""
    code = _dense_code(w, "w")
    if w.numel() != m.rows * m.K:
        raise ValueError(f"w: {w.numel()} elements, m holds {m.rows * m.K}")
    (pw,) = _args((w, "w", 0, w.dtype, True))
    _check(lib().moe_w4_dequantize(m.rows, m.K, code, m.group, m._c(), pw, _raw_stream(stream)),
           "moe_w4_dequantize")


def _w4_args(c: CConfig, w1, w3, w2, ws1, ws3, ws2):
    """The group size and the C structs of a block's 4-bit weights, checked."""
    sh = c.f_shared > 0
    out, group = [], None
    for m, name, rows, K, required in ((w1, "w1", c.E * c.f, c.d, True), (w3, "w3", c.E * c.f, c.d, True),
                                       (w2, "w2", c.E * c.d, c.f, True), (ws1, "ws1", c.f_shared, c.d, sh),
                                       (ws3, "ws3", c.f_shared, c.d, sh), (ws2, "ws2", c.d, c.f_shared, sh)):
        if not required:
            out.append(None)
            continue
        if not isinstance(m, W4Matrix):
            raise TypeError(f"{name} must be a W4Matrix, not {type(m).__name__}")
        if m.K != K or m.rows < rows:
            raise ValueError(f"{name}: {m.rows} rows of {m.K}, needs {rows} rows of {K}")
        if group is not None and m.group != group:
            raise ValueError(f"{name}: group {m.group}, the others have {group}")
        group = m.group
        out.append(m)
    return group, [None if m is None else m._c() for m in out]


def moe_expert_swiglu_w4(cfg, x, perm_src, expert_offsets, w1, w3, w2, x_shared, ws1, ws3, ws2, y_perm, y_shared,
                         workspace, stream=None):
    """moe_expert_swiglu on 4-bit weights (W4Matrix); rows gathered from x by perm_src, or packed if it is None."""
    c = _cfg(cfg)
    R, d, dt, sh = c.T * c.k, c.d, _dt(c), c.f_shared > 0
    px, pp, po, pxs, py, pys, pw = _args(
        (x, "x", (R if perm_src is None else c.T) * d, dt, True), (perm_src, "perm_src", R, _I32, False),
        (expert_offsets, "expert_offsets", c.E + 1, _I32, True), (x_shared, "x_shared", c.T * d, dt, sh),
        (y_perm, "y_perm", R * d, dt, True), (y_shared, "y_shared", c.T * d, dt, sh),
        (workspace, "workspace", 1, _U8, True))
    group, (a1, a3, a2, s1, s3, s2) = _w4_args(c, w1, w3, w2, ws1, ws3, ws2)
    _check(lib().moe_expert_swiglu_w4(ctypes.byref(c), group, px, pp, po, a1, a3, a2, pxs, s1, s3, s2, py, pys, pw,
                                      workspace.numel(), _raw_stream(stream)), "moe_expert_swiglu_w4")


def moe_forward_w4(cfg, x, w_router, bias, w1, w3, w2, ws1, ws3, ws2, y, workspace, stream=None):
    """The block on 4-bit expert weights (W4Matrix); the router's weights are bf16."""
    c = _cfg(cfg)
    dt = _dt(c)
    group, (a1, a3, a2, s1, s3, s2) = _w4_args(c, w1, w3, w2, ws1, ws3, ws2)
    px, pr, pb, py, pw = _args((x, "x", c.T * c.d, dt, True), (w_router, "w_router", c.E * c.d, dt, True),
                               (bias, "bias", c.E, _F32, False), (y, "y", c.T * c.d, dt, True),
                               (workspace, "workspace", 1, _U8, True))
    _check(lib().moe_forward_w4(ctypes.byref(c), group, px, pr, pb, a1, a3, a2, s1, s3, s2, py, pw,
                                workspace.numel(), _raw_stream(stream)), "moe_forward_w4")


# --------------------------------------------------------- orthogonalisation
def make_ortho_config(cfg: Optional[OrthoConfig] = None, **kw) -> COrthoConfig:
    """The C struct of an OrthoConfig, or of one with the given fields."""
    cfg = OrthoConfig(**kw) if cfg is None else cfg
    return COrthoConfig(n=cfg.n, rows=cfg.rows, cols=cfg.cols, dtype=_dtype_code(cfg.dtype), steps=cfg.steps,
                        eps=cfg.eps)


def _ocfg(c) -> COrthoConfig:
    return c if isinstance(c, COrthoConfig) else make_ortho_config(c)


def ortho_workspace_size(cfg) -> int:
    return int(lib().moe_ortho_workspace_size(ctypes.byref(_ocfg(cfg))))


def alloc_ortho_workspace(cfg, device="cuda") -> torch.Tensor:
    n = ortho_workspace_size(cfg)
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_ortho_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _coeffs(c: COrthoConfig, coeffs):
    """The host array of a, b, c per step: None for the default, one triple for
    every step, or a triple for each."""
    if coeffs is None:
        return None
    flat = [float(v) for t in coeffs for v in (t if isinstance(t, (tuple, list)) else (t,))]
    if len(flat) == 3:
        flat *= max(c.steps, 1)
    if len(flat) != 3 * c.steps:
        raise ValueError(f"coeffs: {len(flat)} numbers, expected 3 or {3 * c.steps}")
    return (ctypes.c_float * len(flat))(*flat)


def moe_orthogonalize(cfg, g, o, workspace, coeffs=None, stream=None):
    """Newton-Schulz orthogonalisation of every matrix of g [n, rows, cols] into o (bf16)."""
    c = _ocfg(cfg)
    n = c.n * c.rows * c.cols
    abc = _coeffs(c, coeffs)
    pg, po, pw = _args((g, "g", n, _dt(c), True), (o, "o", n, torch.bfloat16, True),
                       (workspace, "workspace", 1, _U8, True))
    _check(lib().moe_orthogonalize(ctypes.byref(c), abc, pg, po, pw, workspace.numel(), _raw_stream(stream)),
           "moe_orthogonalize")


def moe_muon_step(cfg, g, momentum, weight, workspace, lr: float, mu: float = 0.95, nesterov: bool = True,
                  weight_decay: float = 0.0, scale: float = 1.0, coeffs=None, stream=None):
    """Muon's update in place: momentum (fp32) by g, weight (fp32 or bf16) by the orthogonalised momentum."""
    c = _ocfg(cfg)
    n = c.n * c.rows * c.cols
    code = _dense_code(weight, "weight")
    abc = _coeffs(c, coeffs)
    pg, pm, pw, ps = _args((g, "g", n, _dt(c), True), (momentum, "momentum", n, _F32, True),
                           (weight, "weight", n, weight.dtype, True), (workspace, "workspace", 1, _U8, True))
    _check(lib().moe_muon_step(ctypes.byref(c), abc, pg, pm, pw, code, lr, mu, int(nesterov), weight_decay, scale, ps,
                               workspace.numel(), _raw_stream(stream)), "moe_muon_step")


# ------------------------------------------------------------ residual norms
def make_norm_config(cfg: Optional[NormConfig] = None, **kw) -> CNormConfig:
    """The C struct of a NormConfig, or of one with the given fields."""
    cfg = NormConfig(**kw) if cfg is None else cfg
    return CNormConfig(T=cfg.T, d=cfg.d, dtype=_dtype_code(cfg.dtype), gate_tokens=cfg.gate_tokens, eps=cfg.eps,
                       alpha=cfg.alpha, beta=cfg.beta, w_offset=cfg.w_offset)


def _dtype_code(name: str) -> int:
    if name not in ("f32", "bf16"):
        raise ValueError(f"dtype {name!r}: expected 'f32' or 'bf16'")
    return MOE_DTYPE_F32 if name == "f32" else MOE_DTYPE_BF16


def _ncfg(c) -> CNormConfig:
    return c if isinstance(c, CNormConfig) else make_norm_config(c)


def _gate_elems(c: CNormConfig) -> int:
    return -(-c.T // max(c.gate_tokens, 1)) * c.d


def moe_residual_norm(cfg, h, y, w_post, gate, w_pre, h_out, u, stream=None):
    """h_out = alpha h + beta gate . N(y; w_post) and u = N(h_out; w_pre) in one pass."""
    c = _ncfg(cfg)
    dt, d = _dt(c), c.d
    n = c.T * d
    a = _args((h, "h", n, dt, True), (y, "y", n, dt, False), (w_post, "w_post", d, dt, False),
              (gate, "gate", _gate_elems(c), dt, False), (w_pre, "w_pre", d, dt, False),
              (h_out, "h_out", n, dt, y is not None), (u, "u", n, dt, w_pre is not None))
    _check(lib().moe_residual_norm(ctypes.byref(c), *a, _raw_stream(stream)), "moe_residual_norm")


def norm_backward_workspace_size(cfg) -> int:
    return int(lib().moe_residual_norm_backward_workspace_size(ctypes.byref(_ncfg(cfg))))


def alloc_norm_backward_workspace(cfg, device="cuda") -> torch.Tensor:
    n = norm_backward_workspace_size(cfg)
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_residual_norm_backward_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_residual_norm_backward(cfg, h_out, y, w_post, gate, w_pre, du, dh_out, dh, dy, dw_post, dgate, dw_pre,
                               workspace, stream=None):
    """Gradients of moe_residual_norm, given those of u and of h_out (None: none)."""
    c = _ncfg(cfg)
    dt, d, gates = _dt(c), c.d, _gate_elems(c)
    n = c.T * d
    a = _args((h_out, "h_out", n, dt, w_pre is not None), (y, "y", n, dt, False), (w_post, "w_post", d, dt, False),
              (gate, "gate", gates, dt, False), (w_pre, "w_pre", d, dt, False),
              (du, "du", n, dt, w_pre is not None), (dh_out, "dh_out", n, dt, False), (dh, "dh", n, dt, False),
              (dy, "dy", n, dt, False), (dw_post, "dw_post", d, dt, False), (dgate, "dgate", gates, dt, False),
              (dw_pre, "dw_pre", d, dt, False), (workspace, "workspace", 1, _U8, True))
    _check(lib().moe_residual_norm_backward(ctypes.byref(c), *a, workspace.numel(), _raw_stream(stream)),
           "moe_residual_norm_backward")


def moe_get_device_error(workspace, stream=None) -> int:
    _need_ws(workspace)
    return lib().moe_get_device_error(_ptr(workspace), _stream(stream))


def moe_selftest_wait_timeout(workspace, timeout_ns: int, stream=None):
    _need_ws(workspace)
    _check(lib().moe_selftest_wait_timeout(_ptr(workspace), workspace.numel(), int(timeout_ns),
                                           _stream(stream)), "moe_selftest_wait_timeout")


class MoEBlock:
    """Convenience wrapper holding one block's weights and workspace on the GPU.

    ``forward(x)`` returns a new ``[T, d]`` tensor (shared + routed, no
    residual) computed by ``moe_forward``, or by ``moe_forward_w4`` where the
    expert weights are ``W4Matrix``.

    Calls run on ``stream`` (None: the current one), which comes after the work
    that makes their inputs; tensors that they return are allocated on it. Calls
    of one T share a workspace: they belong on one stream, or are ordered by
    events.
    """

    def __init__(self, cfg: MoEConfig, weights: dict, device="cuda"):
        self.cfg = cfg
        self.w = weights
        self.device = torch.device(device)
        self._ws = {}

    def workspace(self, T: int, stream=None) -> torch.Tensor:
        if T not in self._ws:
            with _allocating_on(stream):
                self._ws[T] = alloc_workspace(make_config(self.cfg, T), self.device)
        return self._ws[T]

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        if out is None:
            with _allocating_on(stream):
                out = torch.empty_like(x)
        w = self.w
        run = moe_forward_w4 if isinstance(w["w1"], W4Matrix) else moe_forward
        run(make_config(self.cfg, T), x, w["w_router"], w.get("bias"), w["w1"], w["w3"], w["w2"],
            w.get("ws1"), w.get("ws3"), w.get("ws2"), out, self.workspace(T, stream), stream)
        return out

    def step(self, h: torch.Tensor, u: torch.Tensor, norm: NormConfig, w_post=None, gate=None, w_pre=None, h_out=None,
             u_out=None, stream=None):
        """One layer of a residual stack: ``(h_out, u_out)`` from the stream h and
        the block's normalised input u. The block runs on u; its output is
        normalised by w_post, gated, scaled and added to the stream
        (``moe_residual_norm``; ``norm`` gives the scales, its T and d are h's),
        and u_out is the next block's input under w_pre (None without one).
        ``h_out`` may be h, ``u_out`` may be u."""
        T, d = h.shape
        y = self.forward(u, stream=stream)
        with _allocating_on(stream):
            if h_out is None:
                h_out = torch.empty_like(h)
            if u_out is None and w_pre is not None:
                u_out = torch.empty_like(h)
        cfg = make_norm_config(dataclasses.replace(norm, T=T, d=d, dtype="f32" if h.dtype == torch.float32 else "bf16"))
        moe_residual_norm(cfg, h, y, w_post, gate, w_pre, h_out, u_out, stream)
        return h_out, u_out
