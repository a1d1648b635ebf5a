"""Python binding of libmoe (include/moe.h): argument marshalling only.

Every function below has the name of the C entry point it calls and takes
torch tensors (or None for a NULL pointer, or an int address) in the C
argument order.  All arithmetic runs in libmoe's CUDA kernels; if the library
is missing this module raises at import time instead of falling back to
anything else.

``MoELayer`` is a small convenience holder: it keeps the weights and one
workspace per stream (allocated with torch) and calls ``moe_forward``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

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


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run token_dispatch_grouped_fp32_gb300.build.build() "
            "(nvcc, sm_103a). There is no fallback path.")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    cfgp = ctypes.POINTER(moe_config_t)
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


def _ptr(t):
    if isinstance(t, torch.Tensor):
        if not t.is_contiguous():
            raise ValueError("tensors passed to libmoe must be contiguous")
        return t.data_ptr()
    if t is None or isinstance(t, int):
        return t
    raise TypeError(f"expected a torch.Tensor, an int address or None, got {type(t)}")


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
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


class MoELayer:
    """Weights of one MoE layer plus reusable workspaces; ``forward`` runs
    ``moe_forward`` on the given (default: current) stream.  Weights: Wr [E, d]
    fp32, W_gate_up [E, d, 2f] and W_down [E, f, d] in the activation dtype,
    optional per-expert logit bias [E] fp32.

    The workspace holds a call's intermediates (logits, routing, permuted
    rows), so two calls in flight at once must not share one: the layer keeps
    a separate workspace for each stream it is called on.  A call with a
    ``stream`` that is not the current one allocates from that stream's pool,
    and neither what it returns nor the tensors given to it go back to a pool
    before both streams are done with them; ordering the two streams is the
    caller's part.  A workspace that a graph was captured with stays allocated as
    long as the layer, also when a longer batch gets a new one.

    ``backward`` runs ``moe_backward`` for the latest ``forward`` on the same
    stream, whose intermediates it finds in that workspace.  It refuses when
    they are not there: after a ``forward`` that failed, when the workspace has
    been replaced by a larger one, when the layer's sizes or modes have changed,
    and for an ``x`` that is not the memory the forward read or has been written
    to since (by torch's count of in-place writes, which views of one tensor
    share; not looked at where the forward was captured in a graph, whose
    replays read ``x`` afresh)."""

    def __init__(self, Wr, W_gate_up, W_down, k, logit_bias=None, renormalize=True,
                 scale_inputs=False):
        self.Wr, self.W_gate_up, self.W_down = Wr, W_gate_up, W_down
        self.logit_bias = logit_bias
        self.E, self.d = Wr.shape
        self.f = W_down.shape[1]
        self.k = int(k)
        self.dtype = W_gate_up.dtype
        self.renormalize = renormalize
        self.scale_inputs = scale_inputs
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
        return torch.cuda.ExternalStream(key) if key else torch.cuda.default_stream()

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
        moe_forward(cfg, x, self.Wr, self.logit_bias, self.W_gate_up, self.W_down, out, ws,
                    stream=key)
        self._tokens[key] = cfg.T
        version = None if self._capturing(ws) else _version(x)
        if _ptr(out) != x.data_ptr():
            self._forwards[key] = (ws, bytes(cfg), x.data_ptr(), version)
        return out

    __call__ = forward

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
        if T and (ran != bytes(cfg) or at != x.data_ptr() or written):
            raise RuntimeError("x is not what the latest forward on this stream read, has been "
                               "written to since, or the layer has changed since")
        _record(side, (x, dout))
        if side is not None:
            _record(torch.cuda.current_stream() if made else side, grads.values())
        ws = self._grown(self._bwd_ws, moe_backward_workspace_size(cfg), stream, key)
        self._capturing(ws, *(() if fwd_ws is None else (fwd_ws,)))
        moe_backward(cfg, x, self.Wr, self.W_gate_up, self.W_down, fwd_ws, dout, grads["x"],
                     grads["Wr"], grads.get("logit_bias"), grads["W_gate_up"], grads["W_down"], ws,
                     stream=key)
        return grads
