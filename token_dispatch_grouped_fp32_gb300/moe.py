"""Python binding of libmoe (include/moe.h): argument marshalling only.

Every function below has the name of the C entry point it calls and takes
torch tensors (or None for a NULL pointer, or an int address) in the C
argument order.  All arithmetic runs in libmoe's CUDA kernels; if the library
is missing this module raises at import time instead of falling back to
anything else.

``MoELayer`` is a small convenience holder: it keeps the weights and one
workspace per stream (allocated with torch) and calls ``moe_forward``;
``AdamW`` holds an optimizer's states and calls ``moe_adamw_step``.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4
MOE_ERR_DEVICE_TIMEOUT = -5
MOE_ERR_BAD_ROUTING = -6
MOE_F32 = 0
MOE_BF16 = 1
MOE_E4M3 = 2
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_GROUP_MAX = 0
MOE_GROUP_TOP2 = 1
ADAMW_BLOCK = 256  # elements under one scale of an 8-bit state


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {_status_name(status)} ({detail})")
        self.status = status


class moe_config_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("f", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale_inputs", ctypes.c_int32)]


# moe_workspace_layout: offset of a region moe_forward does not use
MOE_WS_ABSENT = (1 << (8 * ctypes.sizeof(ctypes.c_size_t))) - 1


class moe_workspace_layout_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("logits", "topk_idx", "topk_w", "counts", "offsets",
                                               "pos", "src_token", "x_perm", "h_perm", "y_perm",
                                               "total")]


class moe_grad_t(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class moe_router_t(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("weight_scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class moe_adamw_tensor_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq",
                                               "exp_avg_scale", "exp_avg_sq_scale", "master")] + \
        [("numel", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
         ("state_dtype", ctypes.c_int32), ("weight_decay", ctypes.c_float)]


class moe_adamw_hyper_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("seed", ctypes.c_uint64),
                ("max_norm", ctypes.c_float), ("stochastic", ctypes.c_int32),
                ("skip_nonfinite", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class moe_adamw_scalars_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("step_size", ctypes.c_float),
                ("inv_sqrt_bc2", ctypes.c_float), ("seed_lo", ctypes.c_uint32),
                ("seed_hi", ctypes.c_uint32), ("reserved", ctypes.c_uint32 * 3)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run token_dispatch_grouped_fp32_gb300.build.build() "
            "(nvcc, sm_103a). There is no fallback path.")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    cfgp, rtp = ctypes.POINTER(moe_config_t), ctypes.POINTER(moe_router_t)
    sig = {
        "moe_status_string": ([st], ctypes.c_char_p),
        "moe_last_error_message": ([], ctypes.c_char_p),
        "moe_workspace_size": ([cfgp], sz),
        "moe_dispatch_workspace_size": ([cfgp], sz),
        "moe_forward_kernel_launches": ([cfgp], st),
        "moe_route": ([cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp], st),
        "moe_route_workspace_size": ([cfgp], sz),
        "moe_route_from_logits": ([cfgp, vp, vp, vp, vp], st),
        "moe_dispatch": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], st),
        "moe_grouped_swiglu": ([cfgp, vp, vp, vp, vp, vp, vp, vp], st),
        "moe_combine": ([cfgp, vp, vp, vp, vp, vp], st),
        "moe_forward": ([cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp], st),
        "moe_forward_host": ([cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], st),
        "moe_combine_backward": ([cfgp] + [vp] * 7, st),
        "moe_dispatch_backward": ([cfgp] + [vp] * 7, st),
        "moe_grouped_swiglu_backward_workspace_size": ([cfgp], sz),
        "moe_grouped_swiglu_backward": ([cfgp] + [vp] * 10 + [sz, vp], st),
        "moe_route_backward_workspace_size": ([cfgp], sz),
        "moe_route_backward": ([cfgp] + [vp] * 12 + [sz, vp], st),
        "moe_backward_workspace_size": ([cfgp], sz),
        "moe_backward": ([cfgp] + [vp] * 5 + [sz] + [vp] * 7 + [sz, vp], st),
        "moe_clip_grad_norm_workspace_size": ([], sz),
        "moe_clip_grad_norm": ([ctypes.POINTER(moe_grad_t), ctypes.c_int64, ctypes.c_float, vp, vp,
                                sz, vp], st),
        "moe_route_scored": ([cfgp, rtp] + [vp] * 8 + [sz, vp], st),
        "moe_route_scored_from_logits": ([cfgp, rtp] + [vp] * 5, st),
        "moe_route_scored_from_logits_backward": ([cfgp, rtp] + [vp] * 6, st),
        "moe_route_scored_backward_workspace_size": ([cfgp, rtp], sz),
        "moe_route_scored_backward": ([cfgp, rtp] + [vp] * 12 + [sz, vp], st),
        "moe_forward_scored": ([cfgp, rtp] + [vp] * 8 + [sz, vp], st),
        "moe_backward_scored_workspace_size": ([cfgp, rtp], sz),
        "moe_backward_scored": ([cfgp, rtp] + [vp] * 5 + [sz] + [vp] * 7 + [sz, vp], st),
        "moe_update_balance_bias": ([vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_float] + [vp] * 3,
                                    st),
        "moe_adamw_scalars": ([ctypes.POINTER(moe_adamw_hyper_t),
                               ctypes.POINTER(moe_adamw_scalars_t)], st),
        "moe_adamw_step": ([ctypes.POINTER(moe_adamw_tensor_t), ctypes.c_int64,
                            ctypes.POINTER(moe_adamw_hyper_t), vp, vp, vp], st),
        "moe_last_device_error": ([vp], st),
        "moe_set_wait_limit_ns": ([ctypes.c_uint64], None),
        "moe_wait_limit_ns": ([], ctypes.c_uint64),
        "moe_workspace_layout": ([cfgp, ctypes.POINTER(moe_workspace_layout_t)], st),
        "moe_debug_inject_wait_timeout": ([ctypes.c_int], None),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def _status_name(status: int) -> str:
    return _lib.moe_status_string(int(status)).decode()


# A call's Python side costs as much as a small kernel: addresses are passed
# as plain ints, and the current stream is read as a raw handle where torch
# has one (2.5 us less a call than through a Stream object).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)
_started = False  # torch has brought up CUDA: the raw calls do


def _ptr(t):
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors passed to libmoe must be contiguous")
        return t.data_ptr()
    if t is None or isinstance(t, int):
        return t
    raise TypeError(f"expected a torch.Tensor, an int address or None, got {type(t)}")


def _stream(stream):
    global _started
    if stream is None:
        if _started:
            return _raw_stream(_raw_device())
        if _raw_stream is not None:
            device = torch.cuda.current_device()
            _started = _raw_device is not None
            return _raw_stream(device)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str, raise_on_error: bool):
    if status != MOE_OK and raise_on_error:
        raise MoEError(status, where, _lib.moe_last_error_message().decode())
    return status


def config(T: int, d: int, E: int, k: int, f: int, dtype=torch.bfloat16,
           renormalize: bool = True, scale_inputs: bool = False) -> moe_config_t:
    if dtype in (torch.bfloat16, "bf16", MOE_BF16):
        act = MOE_BF16
    elif dtype in (torch.float32, "f32", MOE_F32):
        act = MOE_F32
    else:
        act = int(dtype)
    return moe_config_t(int(T), int(d), int(E), int(k), int(f), act, int(bool(renormalize)),
                        int(bool(scale_inputs)))


def moe_status_string(status: int) -> str:
    return _status_name(status)


def moe_last_error_message() -> str:
    return _lib.moe_last_error_message().decode()


def moe_workspace_size(cfg: moe_config_t) -> int:
    return int(_lib.moe_workspace_size(ctypes.byref(cfg)))


def moe_dispatch_workspace_size(cfg: moe_config_t) -> int:
    return int(_lib.moe_dispatch_workspace_size(ctypes.byref(cfg)))


def moe_forward_kernel_launches(cfg: moe_config_t) -> int:
    return int(_lib.moe_forward_kernel_launches(ctypes.byref(cfg)))


def moe_set_wait_limit_ns(ns: int) -> None:
    _lib.moe_set_wait_limit_ns(int(ns))


def moe_wait_limit_ns() -> int:
    return int(_lib.moe_wait_limit_ns())


def moe_workspace_layout(cfg: moe_config_t, raise_on_error=True) -> moe_workspace_layout_t:
    layout = moe_workspace_layout_t()
    _check(_lib.moe_workspace_layout(ctypes.byref(cfg), ctypes.byref(layout)),
           "moe_workspace_layout", raise_on_error)
    return layout


def moe_debug_inject_wait_timeout(enable: bool) -> None:
    _lib.moe_debug_inject_wait_timeout(int(bool(enable)))


def moe_route_workspace_size(cfg: moe_config_t) -> int:
    return int(_lib.moe_route_workspace_size(ctypes.byref(cfg)))


def moe_route(cfg, x, Wr, logit_bias, logits, topk_idx, topk_w, ws=None, ws_bytes=None,
              stream=None, raise_on_error=True):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None or isinstance(ws, int) else ws.numel() * ws.element_size()
    s = _lib.moe_route(ctypes.byref(cfg), _ptr(x), _ptr(Wr), _ptr(logit_bias), _ptr(logits),
                       _ptr(topk_idx), _ptr(topk_w), _ptr(ws), int(ws_bytes), _stream(stream))
    return _check(s, "moe_route", raise_on_error)


def moe_route_from_logits(cfg, logits, topk_idx, topk_w, stream=None, raise_on_error=True):
    s = _lib.moe_route_from_logits(ctypes.byref(cfg), _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
                                   _stream(stream))
    return _check(s, "moe_route_from_logits", raise_on_error)


def moe_dispatch(cfg, topk_idx, topk_w, x, counts, offsets, pos, src_token, x_perm, ws,
                 ws_bytes=None, stream=None, raise_on_error=True):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None or isinstance(ws, int) else ws.numel() * ws.element_size()
    s = _lib.moe_dispatch(ctypes.byref(cfg), _ptr(topk_idx), _ptr(topk_w), _ptr(x), _ptr(counts),
                          _ptr(offsets), _ptr(pos), _ptr(src_token), _ptr(x_perm), _ptr(ws),
                          int(ws_bytes), _stream(stream))
    return _check(s, "moe_dispatch", raise_on_error)


def moe_grouped_swiglu(cfg, x_perm, offsets, W_gate_up, W_down, h_perm, y_perm, stream=None,
                       raise_on_error=True):
    s = _lib.moe_grouped_swiglu(ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(W_gate_up),
                                _ptr(W_down), _ptr(h_perm), _ptr(y_perm), _stream(stream))
    return _check(s, "moe_grouped_swiglu", raise_on_error)


def moe_combine(cfg, y_perm, pos, topk_w, out, stream=None, raise_on_error=True):
    s = _lib.moe_combine(ctypes.byref(cfg), _ptr(y_perm), _ptr(pos), _ptr(topk_w), _ptr(out),
                         _stream(stream))
    return _check(s, "moe_combine", raise_on_error)


def moe_forward(cfg, x, Wr, logit_bias, W_gate_up, W_down, out, ws, ws_bytes=None, stream=None,
                raise_on_error=True):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None or isinstance(ws, int) else ws.numel() * ws.element_size()
    s = _lib.moe_forward(ctypes.byref(cfg), _ptr(x), _ptr(Wr), _ptr(logit_bias), _ptr(W_gate_up),
                         _ptr(W_down), _ptr(out), _ptr(ws), int(ws_bytes), _stream(stream))
    return _check(s, "moe_forward", raise_on_error)


def moe_forward_host(cfg, x_host, Wr, logit_bias, W_gate_up, W_down, out_host, x_dev, out_dev, ws,
                     ws_bytes=None, stream=None, raise_on_error=True):
    if ws_bytes is None:
        ws_bytes = 0 if ws is None or isinstance(ws, int) else ws.numel() * ws.element_size()
    s = _lib.moe_forward_host(ctypes.byref(cfg), _ptr(x_host), _ptr(Wr), _ptr(logit_bias),
                              _ptr(W_gate_up), _ptr(W_down), _ptr(out_host), _ptr(x_dev),
                              _ptr(out_dev), _ptr(ws), int(ws_bytes), _stream(stream))
    return _check(s, "moe_forward_host", raise_on_error)


def _bytes(ws, ws_bytes):
    if ws_bytes is not None:
        return int(ws_bytes)
    return 0 if ws is None or isinstance(ws, int) else ws.numel() * ws.element_size()


def moe_combine_backward(cfg, dout, y_perm, pos, topk_w, dy_perm, dtopk_w, stream=None,
                         raise_on_error=True):
    s = _lib.moe_combine_backward(ctypes.byref(cfg), _ptr(dout), _ptr(y_perm), _ptr(pos),
                                  _ptr(topk_w), _ptr(dy_perm), _ptr(dtopk_w), _stream(stream))
    return _check(s, "moe_combine_backward", raise_on_error)


def moe_dispatch_backward(cfg, dx_perm, pos, topk_w, x, dx, dtopk_w, stream=None,
                          raise_on_error=True):
    s = _lib.moe_dispatch_backward(ctypes.byref(cfg), _ptr(dx_perm), _ptr(pos), _ptr(topk_w),
                                   _ptr(x), _ptr(dx), _ptr(dtopk_w), _stream(stream))
    return _check(s, "moe_dispatch_backward", raise_on_error)


def moe_grouped_swiglu_backward_workspace_size(cfg: moe_config_t) -> int:
    return int(_lib.moe_grouped_swiglu_backward_workspace_size(ctypes.byref(cfg)))


def moe_grouped_swiglu_backward(cfg, x_perm, offsets, W_gate_up, W_down, h_perm, dy_perm, dx_perm,
                                dW_gate_up, dW_down, ws, ws_bytes=None, stream=None,
                                raise_on_error=True):
    s = _lib.moe_grouped_swiglu_backward(
        ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(W_gate_up), _ptr(W_down),
        _ptr(h_perm), _ptr(dy_perm), _ptr(dx_perm), _ptr(dW_gate_up), _ptr(dW_down), _ptr(ws),
        _bytes(ws, ws_bytes), _stream(stream))
    return _check(s, "moe_grouped_swiglu_backward", raise_on_error)


def moe_route_backward_workspace_size(cfg: moe_config_t) -> int:
    return int(_lib.moe_route_backward_workspace_size(ctypes.byref(cfg)))


def moe_route_backward(cfg, x, Wr, logits, topk_idx, topk_w, dtopk_w, dx_in, dlogits, dWr,
                       dlogit_bias, dx, ws, ws_bytes=None, stream=None, raise_on_error=True):
    s = _lib.moe_route_backward(
        ctypes.byref(cfg), _ptr(x), _ptr(Wr), _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
        _ptr(dtopk_w), _ptr(dx_in), _ptr(dlogits), _ptr(dWr), _ptr(dlogit_bias), _ptr(dx), _ptr(ws),
        _bytes(ws, ws_bytes), _stream(stream))
    return _check(s, "moe_route_backward", raise_on_error)


def moe_backward_workspace_size(cfg: moe_config_t) -> int:
    return int(_lib.moe_backward_workspace_size(ctypes.byref(cfg)))


def moe_backward(cfg, x, Wr, W_gate_up, W_down, fwd_ws, dout, dx, dWr, dlogit_bias, dW_gate_up,
                 dW_down, ws, fwd_ws_bytes=None, ws_bytes=None, stream=None, raise_on_error=True):
    s = _lib.moe_backward(
        ctypes.byref(cfg), _ptr(x), _ptr(Wr), _ptr(W_gate_up), _ptr(W_down), _ptr(fwd_ws),
        _bytes(fwd_ws, fwd_ws_bytes), _ptr(dout), _ptr(dx), _ptr(dWr), _ptr(dlogit_bias),
        _ptr(dW_gate_up), _ptr(dW_down), _ptr(ws), _bytes(ws, ws_bytes), _stream(stream))
    return _check(s, "moe_backward", raise_on_error)


def grad_list(grads, outs=None):
    """The moe_grad_t array of moe_clip_grad_norm for bf16 or fp32 tensors and
    where their clipped copies go (default: in place; None in ``outs``: that
    tensor counts in the norm only).  It holds addresses: keep the tensors
    alive, and build it once for buffers that stay where they are."""
    grads = list(grads)
    outs = grads if outs is None else list(outs)
    if len(outs) != len(grads):
        raise ValueError(f"{len(grads)} gradients but {len(outs)} outputs")
    arr = (moe_grad_t * max(1, len(grads)))()
    arr.count = len(grads)
    for a, g, o in zip(arr, grads, outs):
        if g.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"gradients are bf16 or fp32 tensors, not {g.dtype}")
        if o is not None and (o.dtype != g.dtype or o.numel() != g.numel()):
            raise ValueError("a clipped copy has its gradient's dtype and size")
        a.grad, a.out = _ptr(g), _ptr(o)
        a.numel = g.numel()
        a.dtype = MOE_BF16 if g.dtype == torch.bfloat16 else MOE_F32
    return arr


def moe_clip_grad_norm_workspace_size() -> int:
    return int(_lib.moe_clip_grad_norm_workspace_size())


def moe_clip_grad_norm(grads, max_norm, norm, ws, ws_bytes=None, n=None, stream=None,
                       raise_on_error=True):
    """``grads``: from grad_list (n defaults to its length)."""
    n = grads.count if n is None else int(n)
    s = _lib.moe_clip_grad_norm(grads, n, float(max_norm), _ptr(norm), _ptr(ws),
                                _bytes(ws, ws_bytes), _stream(stream))
    return _check(s, "moe_clip_grad_norm", raise_on_error)


def router(score="softmax", groups: int = 1, topk_groups: int | None = None, group_score="max",
           weight_scale: float = 1.0) -> moe_router_t:
    """Scores "softmax" or "sigmoid"; the best ``topk_groups`` (default: all) of
    ``groups`` groups of experts by their "max" or the sum of their "top2"."""
    score = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}.get(score, score)
    group_score = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}.get(group_score, group_score)
    return moe_router_t(int(score), int(groups), int(groups if topk_groups is None else topk_groups),
                        int(group_score), float(weight_scale), 0)


def moe_route_scored(cfg, router, x, Wr, logit_bias, balance_bias, logits, topk_idx, topk_w, ws=None,
                     ws_bytes=None, stream=None, raise_on_error=True):
    s = _lib.moe_route_scored(
        cfg, router, _ptr(x), _ptr(Wr), _ptr(logit_bias),
        _ptr(balance_bias), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(ws),
        _bytes(ws, ws_bytes), _stream(stream))
    return _check(s, "moe_route_scored", raise_on_error)


def moe_route_scored_from_logits(cfg, router, logits, balance_bias, topk_idx, topk_w, stream=None,
                                 raise_on_error=True):
    s = _lib.moe_route_scored_from_logits(cfg, router, _ptr(logits), _ptr(balance_bias),
                                          _ptr(topk_idx), _ptr(topk_w), _stream(stream))
    return _check(s, "moe_route_scored_from_logits", raise_on_error)


def moe_route_scored_from_logits_backward(cfg, router, logits, topk_idx, topk_w, dtopk_w, dlogits,
                                          stream=None, raise_on_error=True):
    s = _lib.moe_route_scored_from_logits_backward(
        cfg, router, _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
        _ptr(dtopk_w), _ptr(dlogits), _stream(stream))
    return _check(s, "moe_route_scored_from_logits_backward", raise_on_error)


def moe_route_scored_backward_workspace_size(cfg: moe_config_t, router: moe_router_t) -> int:
    return int(_lib.moe_route_scored_backward_workspace_size(cfg, router))


def moe_route_scored_backward(cfg, router, x, Wr, logits, topk_idx, topk_w, dtopk_w, dx_in, dlogits,
                              dWr, dlogit_bias, dx, ws, ws_bytes=None, stream=None,
                              raise_on_error=True):
    s = _lib.moe_route_scored_backward(
        cfg, router, _ptr(x), _ptr(Wr), _ptr(logits), _ptr(topk_idx),
        _ptr(topk_w), _ptr(dtopk_w), _ptr(dx_in), _ptr(dlogits), _ptr(dWr), _ptr(dlogit_bias),
        _ptr(dx), _ptr(ws), _bytes(ws, ws_bytes), _stream(stream))
    return _check(s, "moe_route_scored_backward", raise_on_error)


def moe_forward_scored(cfg, router, x, Wr, logit_bias, balance_bias, W_gate_up, W_down, out, ws,
                       ws_bytes=None, stream=None, raise_on_error=True):
    s = _lib.moe_forward_scored(
        cfg, router, _ptr(x), _ptr(Wr), _ptr(logit_bias),
        _ptr(balance_bias), _ptr(W_gate_up), _ptr(W_down), _ptr(out), _ptr(ws),
        _bytes(ws, ws_bytes), _stream(stream))
    return _check(s, "moe_forward_scored", raise_on_error)


def moe_backward_scored_workspace_size(cfg: moe_config_t, router: moe_router_t) -> int:
    return int(_lib.moe_backward_scored_workspace_size(cfg, router))


def moe_backward_scored(cfg, router, x, Wr, W_gate_up, W_down, fwd_ws, dout, dx, dWr, dlogit_bias,
                        dW_gate_up, dW_down, ws, fwd_ws_bytes=None, ws_bytes=None, stream=None,
                        raise_on_error=True):
    s = _lib.moe_backward_scored(
        cfg, router, _ptr(x), _ptr(Wr), _ptr(W_gate_up), _ptr(W_down),
        _ptr(fwd_ws), _bytes(fwd_ws, fwd_ws_bytes), _ptr(dout), _ptr(dx), _ptr(dWr),
        _ptr(dlogit_bias), _ptr(dW_gate_up), _ptr(dW_down), _ptr(ws), _bytes(ws, ws_bytes),
        _stream(stream))
    return _check(s, "moe_backward_scored", raise_on_error)


def moe_update_balance_bias(counts, rate, balance_bias, imbalance=None, layers=None, E=None,
                            stream=None, raise_on_error=True):
    """``counts`` [layers, E] or [E] int32, ``balance_bias`` of the same shape
    fp32, ``imbalance`` [layers] fp32 or None (``layers`` and ``E`` are taken
    from counts where they are not given)."""
    if E is None:
        shape = counts.shape
        E, layers = shape[-1], counts.numel() // max(1, shape[-1])
        if counts.dtype != torch.int32 or balance_bias.dtype != torch.float32 \
                or balance_bias.shape != shape:
            raise ValueError("counts are int32, the balance bias fp32 of the same shape")
        if imbalance is not None and (imbalance.dtype != torch.float32
                                      or imbalance.numel() != layers):
            raise ValueError("the imbalance is fp32, one value a layer")
    s = _lib.moe_update_balance_bias(_ptr(counts), int(layers), int(E), float(rate),
                                     _ptr(balance_bias), _ptr(imbalance), _stream(stream))
    return _check(s, "moe_update_balance_bias", raise_on_error)


def _on_current(device):
    """Refuses tensors that the current device's kernels are not to touch."""
    if device is not None and (device.type != "cuda"
                               or device.index != torch.cuda.current_device()):
        raise ValueError(f"the tensors are on {device}, not on the current GPU")


def adamw_list(tensors):
    """The moe_adamw_tensor_t array of moe_adamw_step.  ``tensors``: dicts of
    "param" and "grad" (bf16 or fp32), "exp_avg" and "exp_avg_sq" (fp32, or
    float8_e4m3fn beside "exp_avg_scale" and "exp_avg_sq_scale", fp32, one for
    256 elements), and optionally "master" (fp32) and "weight_decay".  All are on
    one device, and none that a step writes overlaps another.  It holds
    addresses: keep the tensors alive, and build it once for buffers that stay
    where they are."""
    tensors = list(tensors)
    rows = [_adamw_row(**t) for t in tensors]
    devices = {t["param"].device for t in tensors}
    if len(devices) > 1:
        raise ValueError(f"the tensors are on one device, not on {devices}")
    ends = {}  # of what a step writes, by its start
    written = 0
    for p, _, m, v, ms, rs, master, n, kind, _, state, _ in rows:
        if n == 0:
            continue
        ends[p] = p + (4 * n if kind == MOE_F32 else 2 * n)
        at = 4 * n if state == MOE_F32 else n
        ends[m] = m + at
        ends[v] = v + at
        written += 3
        if state != MOE_F32:
            blocks = -(-n // ADAMW_BLOCK)
            ends[ms] = ms + 4 * blocks
            ends[rs] = rs + 4 * blocks
            written += 2
        if master is not None:
            ends[master] = master + 4 * n
            written += 1
    starts = sorted(ends)
    if len(starts) != written or any(ends[a] > b for a, b in zip(starts, starts[1:])):
        raise ValueError("two tensors that a step writes overlap")
    arr = (moe_adamw_tensor_t * max(1, len(rows)))(*rows)
    arr.count, arr.device = len(rows), devices.pop() if devices else None
    return arr


_ADAMW_TYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
_STATE_TYPES = {torch.float32: MOE_F32, torch.float8_e4m3fn: MOE_E4M3}


def _adamw_row(param, grad, exp_avg, exp_avg_sq, exp_avg_scale=None, exp_avg_sq_scale=None,
               master=None, weight_decay=0.0):
    n, device = param.numel(), param.device
    kind, grad_kind = _ADAMW_TYPES.get(param.dtype), _ADAMW_TYPES.get(grad.dtype)
    state = _STATE_TYPES.get(exp_avg.dtype)
    if kind is None or grad_kind is None:
        raise TypeError(f"parameters and gradients are bf16 or fp32, not {param.dtype}, {grad.dtype}")
    if state is None or exp_avg_sq.dtype != exp_avg.dtype:
        raise TypeError(f"both states are fp32 or float8_e4m3fn, not {exp_avg.dtype}, "
                        f"{exp_avg_sq.dtype}")
    for x in (grad, exp_avg, exp_avg_sq):
        if x.numel() != n:
            raise ValueError("a gradient and its states have the parameter's size")
        if x.device != device:
            raise ValueError("a parameter, its gradient and its states are on one device")
    if master is not None and (kind != MOE_BF16 or master.dtype != torch.float32
                               or master.numel() != n or master.device != device):
        raise ValueError("a master copy is an fp32 tensor of a bf16 parameter's size")
    if state == MOE_F32:
        if exp_avg_scale is not None or exp_avg_sq_scale is not None:
            raise ValueError("scales beside fp32 states")
    else:
        for s in (exp_avg_scale, exp_avg_sq_scale):
            if s is None or s.dtype != torch.float32 or s.numel() != -(-n // ADAMW_BLOCK) \
                    or s.device != device:
                raise ValueError("8-bit states have an fp32 scale for 256 elements")
    return (_ptr(param), _ptr(grad), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(exp_avg_scale),
            _ptr(exp_avg_sq_scale), _ptr(master), n, kind, grad_kind, state, float(weight_decay))


def adamw_hyper(lr, beta1=0.9, beta2=0.95, eps=1e-8, step=1, seed=0, max_norm=0.0,
                stochastic=False, skip_nonfinite=False) -> moe_adamw_hyper_t:
    return moe_adamw_hyper_t(float(lr), float(beta1), float(beta2), float(eps), int(step),
                             int(seed) & (2 ** 64 - 1), float(max_norm), int(bool(stochastic)),
                             int(bool(skip_nonfinite)), 0)


def moe_adamw_scalars(hyper, raise_on_error=True) -> moe_adamw_scalars_t:
    out = moe_adamw_scalars_t()
    _check(_lib.moe_adamw_scalars(hyper, ctypes.byref(out)), "moe_adamw_scalars",
           raise_on_error)
    return out


def moe_adamw_step(tensors, hyper, norm=None, scalars=None, n=None, stream=None,
                   raise_on_error=True):
    """``tensors``: from adamw_list (n defaults to its length); ``norm``: from
    moe_clip_grad_norm, or None; ``scalars``: device memory with a
    moe_adamw_scalars_t, or None."""
    n = tensors.count if n is None else int(n)
    _on_current(getattr(tensors, "device", None))
    s = _lib.moe_adamw_step(tensors, n, hyper, _ptr(norm), _ptr(scalars),
                            _stream(stream))
    return _check(s, "moe_adamw_step", raise_on_error)


def moe_last_device_error(stream=None, raise_on_error=True):
    s = _lib.moe_last_device_error(_stream(stream))
    return _check(s, "moe_last_device_error", raise_on_error)


def _version(x):
    """torch's count of the in-place writes to x (inference tensors have none)."""
    return None if x.is_inference() else x._version


def _allocating_on(side):
    return contextlib.nullcontext() if side is None else torch.cuda.stream(side)


def _record(side, tensors):
    """Keeps the tensors' memory from its pool until `side` is done with it."""
    if side is not None:
        for t in tensors:
            if isinstance(t, torch.Tensor):
                t.record_stream(side)


class _Turns:
    """The bf16 layer calls of one device.  Those that take the GPU alone (see _alone)
    run beside no other, whatever streams they are queued on: their stream waits for the
    end of what other calls' streams hold, and a later call's for theirs.  (Two calls of
    one such shape side by side on two streams have, seldom, not ended: see moe.h on
    streams.)  A call that is being captured in a graph waits for none, and none for it."""

    def __init__(self):
        self.lock = threading.Lock()
        self.last = None  # handle of the stream of the latest call that ran alone
        # that stream and those with calls behind it; an event at the latest one's end
        # where the stream may be gone by the time that it is waited for
        self.ends = {}
        self.kept = set()  # handles that torch keeps to the program's end

    def begin(self, key, alone):
        """Orders stream `key` for a call on it; False: it is being captured."""
        if alone:
            follow = [k for k in self.ends if k != key]
        else:
            follow = [] if self.last is None or key in self.ends else [self.last]
        if not follow:
            return True
        to = _torch_stream(key)
        if _capturing_on(to):
            return False
        for k in follow:
            event = self.ends[k]
            if event is None:
                side = _torch_stream(k)
                if _capturing_on(side):
                    raise RuntimeError("the stream of an earlier layer call is being captured: a call on "
                                       "another stream cannot be ordered behind it")
                event = side.record_event()
            to.wait_event(event)
        return True

    def end(self, stream, key, alone):
        event = None
        if not self.keeps(stream, key):
            side = _torch_stream(key)
            if _capturing_on(side):
                return
            event = side.record_event()
        if alone:
            self.last = key
            self.ends.clear()
        self.ends[key] = event

    def keeps(self, stream, key):
        """Whether torch keeps the stream (its default and pooled ones)."""
        if key in self.kept:
            return True
        if stream is None:
            stream = torch.cuda.current_stream()
        kept = key == 0 or isinstance(stream, torch.cuda.Stream) and stream.stream_id != key
        if kept:
            self.kept.add(key)
        return kept


class _Turn:
    """with _Turn(turns, stream, key, alone): the launches of one call."""

    def __init__(self, *call):
        self.turns, *self.call = call

    def __enter__(self):
        self.turns.lock.acquire()
        try:
            self.counts = self.turns.begin(*self.call[1:])
        except BaseException:
            self.turns.lock.release()
            raise

    def __exit__(self, *exc):
        try:
            if self.counts:
                self.turns.end(*self.call)
        finally:
            self.turns.lock.release()


_turns = collections.defaultdict(_Turns)  # by device index
_MOST_STREAMS = 64


def _torch_stream(key):
    return torch.cuda.ExternalStream(key) if key else torch.cuda.default_stream()


def _capturing_on(stream):
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _alone(cfg):
    """Calls that moe.h says to order."""
    E, P = cfg.E, cfg.T * cfg.k
    return E >= 64 or 64 * E <= P < 512 * E


class MoELayer:
    """Weights of one MoE layer plus reusable workspaces; ``forward`` runs
    ``moe_forward`` on the given (default: current) stream.  Weights: Wr [E, d]
    fp32, W_gate_up [E, d, 2f] and W_down [E, f, d] in the activation dtype,
    optional per-expert logit bias [E] fp32.  ``router``: other scores than
    softmax and top-k alone (from ``router()``), with an optional balance bias [E] fp32, which
    ``update_balance_bias`` moves.

    The workspace holds a call's intermediates (logits, routing, permuted
    rows), so two calls in flight at once must not share one: the layer keeps
    a separate workspace for each stream it is called on.  A call with a
    ``stream`` that is not the current one allocates from that stream's pool,
    and neither what it returns nor the tensors given to it go back to a pool
    before both streams are done with them; ordering the two streams is the
    caller's part.  With bf16 weights, and E >= 64 or 64 <= T k / E < 512, a call runs
    beside no other bf16 layer's on the GPU, whatever streams they are queued on;
    replays of captured calls are the caller's to order.  A workspace that a graph was captured
    with stays allocated as long as the layer, also when a longer batch gets a new
    one.

    ``backward`` runs ``moe_backward`` for the latest ``forward`` on the same
    stream, whose intermediates it finds in that workspace.  It refuses when
    they are not there: after a ``forward`` that failed, when the workspace has
    been replaced by a larger one, when the layer's sizes or modes have changed,
    and for an ``x`` that is not the memory the forward read or has been written
    to since (by torch's count of in-place writes, which views of one tensor
    share; not looked at where the forward was captured in a graph, whose
    replays read ``x`` afresh)."""

    def __init__(self, Wr, W_gate_up, W_down, k, logit_bias=None, renormalize=True,
                 scale_inputs=False, router=None, balance_bias=None):
        if balance_bias is not None:
            if router is None:
                raise ValueError("a balance bias needs a router (moe.router())")
            if balance_bias.shape != Wr.shape[:1] or balance_bias.dtype != torch.float32 \
                    or balance_bias.device != Wr.device:
                raise ValueError(f"the balance bias is [{Wr.shape[0]}] fp32 on {Wr.device}")
        self.Wr, self.W_gate_up, self.W_down = Wr, W_gate_up, W_down
        self.logit_bias = logit_bias
        self.E, self.d = Wr.shape
        self.f = W_down.shape[1]
        self.k = int(k)
        self.dtype = W_gate_up.dtype
        self.renormalize = renormalize
        self.scale_inputs = scale_inputs
        self.router, self.balance_bias = router, balance_bias
        self._ws = {}  # stream handle -> workspace
        self._bwd_ws = {}  # the same for the backward pass
        self._tokens = {}  # stream handle -> tokens of its latest forward
        self._forwards = {}  # ... and its workspace, sizes and x
        self._captured = {}  # workspaces in captured graphs: kept with the layer

    def config(self, T: int) -> moe_config_t:
        return config(T, self.d, self.E, self.k, self.f, self.dtype, self.renormalize,
                      self.scale_inputs)

    def workspace(self, T: int, stream=None):
        """The workspace for calls on `stream` (default: the current stream),
        grown to moe_workspace_size for T tokens when needed.  A workspace that
        grows is a new one: the latest forward's intermediates are gone."""
        ws = self._forward_ws(self.config(T), stream, _stream(stream))
        self._capturing(ws)
        return ws

    def _forward_ws(self, cfg, stream, key):
        kept = self._ws.get(key)
        ws = self._grown(self._ws, moe_workspace_size(cfg), stream, key)
        if ws is not kept:
            self._forget(key)
        return ws

    def _forget(self, key):
        self._tokens.pop(key, None)
        self._forwards.pop(key, None)

    def _grown(self, kept, need, stream, key):
        ws = kept.get(key)
        if ws is None or ws.numel() < need:
            with _allocating_on(self._other(stream, key)):
                ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.Wr.device)
            kept[key] = ws
        return ws

    def _capturing(self, *workspaces):
        """Whether a graph is being captured: it will hold these addresses."""
        if not (workspaces[0].is_cuda and torch.cuda.is_current_stream_capturing()):
            return False
        for ws in workspaces:
            self._captured[ws.data_ptr()] = ws
        return True

    def _other(self, stream, key):
        """`stream` (of handle key) for torch, or None where it is the current one."""
        if stream is None or not self.Wr.is_cuda or key == _stream(None):
            return None
        if isinstance(stream, torch.cuda.Stream):
            return stream
        return _torch_stream(key)

    def _turn(self, stream, key, cfg):
        w = self.W_gate_up
        if not w.is_cuda or w.dtype != torch.bfloat16:
            return contextlib.nullcontext()
        turns = _turns[w.device.index]
        # (a call behind all streams also ends the record of them: streams that come and go)
        return _Turn(turns, stream, key, _alone(cfg) or len(turns.ends) >= _MOST_STREAMS)

    def forward(self, x, out=None, stream=None):
        key, cfg = _stream(stream), self.config(x.shape[0])
        side, given = self._other(stream, key), (x, out)
        if out is None:
            with _allocating_on(side):
                out = torch.empty_like(x)
            if side is not None:
                _record(torch.cuda.current_stream(), (out,))
        _record(side, given)
        ws = self._forward_ws(cfg, stream, key)
        self._forget(key)  # until all of its kernels are launched
        with self._turn(stream, key, cfg):
            if self.router is None:
                moe_forward(cfg, x, self.Wr, self.logit_bias, self.W_gate_up, self.W_down, out, ws,
                            stream=key)
            else:
                moe_forward_scored(cfg, self.router, x, self.Wr, self.logit_bias, self.balance_bias,
                                   self.W_gate_up, self.W_down, out, ws, stream=key)
        self._tokens[key] = cfg.T
        version = None if self._capturing(ws) else _version(x)
        if _ptr(out) != x.data_ptr():
            self._forwards[key] = (ws, self._modes(cfg), x.data_ptr(), version)
        return out

    __call__ = forward

    def _modes(self, cfg):
        return bytes(cfg) if self.router is None else bytes(cfg) + bytes(self.router)

    def update_balance_bias(self, rate, imbalance=None, stream=None):
        """Moves the balance bias by ``rate`` against the loads that the latest
        ``forward`` on this stream dispatched; ``imbalance`` [1] fp32 (optional)
        takes their largest over their mean."""
        key = _stream(stream)
        T, ws = self._tokens.get(key), self._ws.get(key)
        if self.balance_bias is None or not T or ws is None:
            raise RuntimeError("no balance bias, or no forward of any tokens on this stream")
        if imbalance is not None and (imbalance.dtype != torch.float32 or imbalance.numel() != 1
                                      or imbalance.device != self.Wr.device):
            raise ValueError(f"the imbalance is one fp32 value on {self.Wr.device}")
        _on_current(self.Wr.device)
        side = self._other(stream, key)
        _record(side, (self.balance_bias, imbalance))
        self._capturing(ws)
        at = moe_workspace_layout(self.config(T)).counts
        moe_update_balance_bias(ws.data_ptr() + at, rate, self.balance_bias, imbalance, layers=1,
                                E=self.E, stream=key)

    def backward(self, x, dout, grads=None, stream=None):
        """Gradients of <out, dout> for the latest ``forward(x)`` on this
        stream: a dict of "x", "Wr", "W_gate_up", "W_down" and, with a logit
        bias, "logit_bias".  ``grads``: such a dict of buffers to write into
        (a training loop keeps one)."""
        if x.shape[1] != self.d or x.dtype != self.dtype or dout.shape != x.shape \
                or dout.dtype != x.dtype:
            raise ValueError(f"x and dout are [T, {self.d}] {self.dtype}, not {tuple(x.shape)} "
                             f"{x.dtype} and {tuple(dout.shape)} {dout.dtype}")
        if x.device != self.Wr.device or dout.device != x.device:
            raise ValueError(f"x is on device {x.device} and dout on {dout.device}, the layer on "
                             f"{self.Wr.device}")
        key, T = _stream(stream), x.shape[0]
        if T and self._tokens.get(key) != T:
            raise RuntimeError(f"backward of {T} tokens, but the latest forward on this stream had "
                               f"{self._tokens.get(key)}")
        cfg = self.config(T)
        like = {"x": x, "Wr": self.Wr, "W_gate_up": self.W_gate_up, "W_down": self.W_down}
        if self.logit_bias is not None:
            like["logit_bias"] = self.logit_bias
        side, made = self._other(stream, key), grads is None
        if made:
            with _allocating_on(side):
                grads = {n: torch.empty_like(t) for n, t in like.items()}
        shapes = {n: (t.shape, t.dtype) for n, t in like.items()}
        shapes["logit_bias"] = (self.Wr.shape[:1], torch.float32)  # written if given
        for n, (shape, dtype) in shapes.items():
            g = grads.get(n)
            if g is None and n == "logit_bias":
                continue
            if g is None or g.shape != shape or g.dtype != dtype or g.device != x.device:
                raise ValueError(f"the gradient of {n} is {tuple(shape)} {dtype} on {x.device}")
        fwd_ws, ran, at, version = self._forwards.get(key, (None,) * 4)
        written = version is not None and _version(x) not in (None, version)
        if T and (ran != self._modes(cfg) or at != x.data_ptr() or written):
            raise RuntimeError("x is not what the latest forward on this stream read, has been "
                               "written to since, or the layer has changed since")
        _record(side, (x, dout))
        if side is not None:
            _record(torch.cuda.current_stream() if made else side, grads.values())
        need = moe_backward_workspace_size(cfg) if self.router is None else \
            moe_backward_scored_workspace_size(cfg, self.router)
        ws = self._grown(self._bwd_ws, need, stream, key)
        self._capturing(ws, *(() if fwd_ws is None else (fwd_ws,)))
        args = (x, self.Wr, self.W_gate_up, self.W_down, fwd_ws, dout, grads["x"], grads["Wr"],
                grads.get("logit_bias"), grads["W_gate_up"], grads["W_down"], ws)
        with self._turn(stream, key, cfg):
            if self.router is None:
                moe_backward(cfg, *args, stream=key)
            else:
                moe_backward_scored(cfg, self.router, *args, stream=key)
        return grads


class AdamW:
    """moe_adamw_step for a list of parameters and of the gradient buffers that
    a training loop keeps: their states, and the list of addresses, built once (about
    3.5 us a tensor).  The steps read these buffers and nothing else: a parameter's
    .grad is not looked at, so gradients that arrive in new tensors are copied there.

    ``bits``: 32 or 8, of the states.  ``master``: fp32 copies of the bf16
    parameters; without them the bf16 values are rounded stochastically.
    ``max_norm``: the gradients count as clipped to this global norm (their
    buffers keep what they hold), which ``norm`` has after a step; a step whose
    norm is not finite is counted, but leaves everything as it was.  ``weight_decay``: one number, or one a
    parameter.  ``lr`` may be changed between steps.

    In a captured graph (``capturable``) a step reads its number, lr and seed from
    device memory: call ``advance()`` before every replay, on the replay's stream.

    A step's tensors, the given ones too, do not go back to a pool before the stream of
    the step is done with them; ordering that stream behind what wrote them, and a graph's
    replays, is the caller's part (keep the optimizer as long as a graph of its steps)."""

    def __init__(self, params, grads, lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, bits=32,
                 master=True, max_norm=None, seed=0, capturable=False):
        params, grads = list(params), list(grads)
        if len(params) != len(grads) or not params:
            raise ValueError(f"{len(params)} parameters but {len(grads)} gradients")
        if bits not in (8, 32):
            raise ValueError("states have 8 or 32 bits")
        wd = list(weight_decay) if isinstance(weight_decay, (list, tuple)) \
            else [weight_decay] * len(params)
        if len(wd) != len(params):
            raise ValueError(f"{len(wd)} weight decays for {len(params)} parameters")
        self.lr, self.betas, self.eps, self.seed, self.steps = lr, betas, eps, int(seed), 0
        self.max_norm, self.stochastic = max_norm, not master
        self.tensors, device = [], params[0].device
        for p, g, d in zip(params, grads, wd):
            if p.device != device:
                raise ValueError(f"parameters on {p.device} and {device}")
            t = {"param": p, "grad": g, "weight_decay": d}
            kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
            for n in ("exp_avg", "exp_avg_sq"):
                t[n] = torch.zeros(p.numel(), dtype=torch.uint8 if bits == 8 else kind,
                                   device=device).view(kind)
                if bits == 8:
                    t[n + "_scale"] = torch.zeros(-(-p.numel() // ADAMW_BLOCK), device=device)
            if master and p.dtype == torch.bfloat16:
                t["master"] = p.detach().float()
            self.tensors.append(t)
        self._list = adamw_list(self.tensors)
        self.norm = self._ws = self._scalars = None
        if max_norm is not None:
            self._clip = grad_list(grads, [None] * len(grads))
            self._ws = torch.empty(moe_clip_grad_norm_workspace_size(), dtype=torch.uint8,
                                   device=device)
            self.norm = torch.zeros((), device=device)
        if capturable:
            self._scalars = torch.zeros(ctypes.sizeof(moe_adamw_scalars_t), dtype=torch.uint8,
                                        device=device)
        # streams that the memory of all of these does not go back to a pool before
        self._streams = {_stream(None)} if device.type == "cuda" else set()

    def _used_here(self):
        """On the current stream: the tensors' memory stays until it is done with them."""
        key = _stream(None)
        if key not in self._streams:
            here = torch.cuda.current_stream()
            for t in self.tensors:
                _record(here, t.values())
            _record(here, (self.norm, self._ws, self._scalars))
            self._streams.add(key)

    def _hyper(self):
        # (another seed every step: the one given, and the step's number)
        return adamw_hyper(self.lr, *self.betas, self.eps, max(1, self.steps),
                           (self.seed << 32) + self.steps, self.max_norm or 0.0, self.stochastic,
                           skip_nonfinite=self.max_norm is not None)

    def advance(self):
        """Counts a step; capturable: what its replay reads, on the current stream."""
        self.steps += 1
        if self._scalars is not None:
            self._used_here()
            raw = torch.frombuffer(bytearray(bytes(moe_adamw_scalars(self._hyper()))),
                                   dtype=torch.uint8)
            self._scalars.copy_(raw, non_blocking=True)

    def step(self, stream=None):
        """One step on the given (default: current) stream."""
        side = stream
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            side = torch.cuda.ExternalStream(int(stream)) if int(stream) \
                else torch.cuda.default_stream()
        with _allocating_on(side):
            _on_current(self._list.device)
            self._used_here()
            if torch.cuda.is_current_stream_capturing():
                if self._scalars is None:
                    raise RuntimeError("a step is captured with capturable=True")
            else:
                self.advance()
            if self.max_norm is not None:
                moe_clip_grad_norm(self._clip, self.max_norm, self.norm, self._ws)
            moe_adamw_step(self._list, self._hyper(), self.norm, self._scalars)
