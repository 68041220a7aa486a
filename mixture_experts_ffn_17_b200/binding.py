"""ctypes binding of libmoe (include/moe.h): argument marshalling only.

Every function takes torch CUDA tensors, passes their data pointers and the
current CUDA stream to the C entry point of the same name, and raises
MoeError on a non-OK status.  All computation happens in the library's
kernels; nothing here computes on the host.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, \
    MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_DEVICE_BOUNDS = range(7)
MOE_BF16, MOE_E4M3, MOE_F32, MOE_MXFP4 = 0, 1, 2, 3
MOE_FEW_MAX_TOKENS = 16
MOE_GRAD_MAX_TENSORS = 1024
MOE_ROUTE_TOPK_SOFTMAX, MOE_ROUTE_SIGMOID_GROUP = 0, 1

EXPORTED = ("moe_workspace_size", "moe_router_topk", "moe_permute", "moe_grouped_swiglu", "moe_combine",
            "moe_forward", "moe_forward_profiled", "moe_check_device_status", "moe_status_string", "moe_version",
            "moe_permute_noalloc", "moe_router_topk_limited", "moe_expert_utilisation", "moe_forward_ep",
            "moe_forward_launches", "moe_combine_backward", "moe_router_backward", "moe_backward_workspace_size",
            "moe_backward", "moe_shared_expert", "moe_ep_regroup_layout", "moe_gather_rows", "moe_forward_train",
            "moe_backward_saved", "moe_few_workspace_size", "moe_forward_few", "moe_mx_quantise",
            "moe_mx_quantise_weights", "moe_mx_dequantise", "moe_mx_product_workspace_size", "moe_mx_grouped_product",
            "moe_grad_workspace_size", "moe_grad_norm", "moe_grad_clip")
NUM_STAGE_EVENTS = 6
STAGES = ("router", "dispatch", "experts_up", "experts_down", "combine")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("shared_inter", ctypes.c_int32), ("route", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32), ("group_topn", ctypes.c_int32),
                ("route_scale", ctypes.c_float), ("w_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32)]


class MoeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


def make_shape(T, d, E, k, inter, shared_inter, route=0, n_group=1, topk_group=1, group_topn=2,
               route_scale=1.0, w_dtype=MOE_BF16, y_dtype=MOE_F32) -> MoeShape:
    return MoeShape(int(T), int(d), int(E), int(k), int(inter), int(shared_inter), int(route), int(n_group),
                    int(topk_group), int(group_topn), float(route_scale), int(w_dtype), int(y_dtype))


def shape_of(cfg, y_dtype=MOE_F32) -> MoeShape:
    """MoeShape of a workloads.Config."""
    return make_shape(cfg.T, cfg.d, cfg.E, cfg.k, cfg.inter, cfg.shared_inter, cfg.route, cfg.n_group,
                      cfg.topk_group, cfg.group_topn, cfg.route_scale, MOE_E4M3 if cfg.fp8 else MOE_BF16, y_dtype)


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so; raises when it is missing (there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmoe.so not built ({LIB_PATH}); run `python -m mixture_experts_ffn_17_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, S, sz = ctypes.c_void_p, ctypes.POINTER(MoeShape), ctypes.c_size_t
        L.moe_workspace_size.argtypes = [S]
        L.moe_workspace_size.restype = sz
        L.moe_router_topk.argtypes = [S, P, P, P, P, P, P, P, sz, P]
        L.moe_permute.argtypes = [S, P, P, P, P, P, P, P, P, sz, P]
        L.moe_permute_noalloc.argtypes = [S, P, P, P, P, P, P, P, P]
        L.moe_router_topk_limited.argtypes = [S, P, P, P, P, P, P, P, sz, P]
        L.moe_router_topk_limited.restype = ctypes.c_int
        L.moe_expert_utilisation.argtypes = [S, P, P, P, P]
        L.moe_expert_utilisation.restype = ctypes.c_int
        L.moe_permute_noalloc.restype = ctypes.c_int
        L.moe_grouped_swiglu.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.moe_combine.argtypes = [S, P, P, P, P, P, P]
        L.moe_combine_backward.argtypes = [S, P, P, P, P, P, P, P]
        L.moe_router_backward.argtypes = [S, P, P, P, P, P, P]
        L.moe_forward.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.moe_forward_profiled.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, sz, P, P]
        I = ctypes.c_int
        L.moe_forward_ep.argtypes = [S, I, I, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.moe_forward_launches.argtypes = [S]
        L.moe_forward_launches.restype = ctypes.c_int
        L.moe_shared_expert.argtypes = [S, P, P, P, P, P, P, sz, P]
        L.moe_ep_regroup_layout.argtypes = [ctypes.c_int, ctypes.c_int, P, P, P, P, P]
        L.moe_gather_rows.argtypes = [P, P, ctypes.c_int64, ctypes.c_int, P, P]
        L.moe_backward_workspace_size.argtypes = [S]
        L.moe_backward_workspace_size.restype = sz
        L.moe_backward.argtypes = [S] + [P] * 18 + [P, sz, P]
        L.moe_forward_train.argtypes = [S] + [P] * 10 + [P, sz, P]
        L.moe_backward_saved.argtypes = [S] + [P] * 17 + [P, sz, P]
        L.moe_few_workspace_size.argtypes = [S]
        L.moe_few_workspace_size.restype = sz
        L.moe_forward_few.argtypes = [S] + [P] * 16 + [P, sz, P]
        i64 = ctypes.c_int64
        L.moe_mx_quantise.argtypes = [P, P, I, i64, I, i64, P, P, P]
        L.moe_mx_quantise_weights.argtypes = [P, I, I, I, I, P, P, P]
        L.moe_mx_dequantise.argtypes = [P, P, i64, I, P, I, P]
        L.moe_mx_product_workspace_size.argtypes = [i64, I]
        L.moe_mx_product_workspace_size.restype = sz
        L.moe_mx_grouped_product.argtypes = [i64, I, I, I, P, P, P, P, P, P, I, P, sz, P]
        L.moe_grad_workspace_size.argtypes = [I]
        L.moe_grad_workspace_size.restype = sz
        L.moe_grad_norm.argtypes = [P, I, P, P, sz, P]
        L.moe_grad_clip.argtypes = [P, I, ctypes.c_float, P, P, sz, P]
        L.moe_check_device_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_uint32)]
        for fn in ("moe_router_topk", "moe_permute", "moe_grouped_swiglu", "moe_combine", "moe_combine_backward",
                   "moe_router_backward", "moe_forward",
                   "moe_forward_profiled", "moe_forward_ep", "moe_backward", "moe_shared_expert", "moe_ep_regroup_layout", "moe_gather_rows",
                   "moe_forward_train", "moe_backward_saved", "moe_forward_few", "moe_mx_quantise",
                   "moe_mx_quantise_weights", "moe_mx_dequantise", "moe_mx_grouped_product", "moe_grad_norm",
                   "moe_grad_clip", "moe_check_device_status"):
            getattr(L, fn).restype = ctypes.c_int
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_version.argtypes = []
        L.moe_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def workspace_size(shape: MoeShape) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(shape)))


def alloc_workspace(shape: MoeShape, device="cuda") -> torch.Tensor:
    n = workspace_size(shape)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def router_topk(shape, x, Wg, bias, topk_idx, topk_w, logits, ws, stream=None):
    _check(lib().moe_router_topk(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(topk_idx), _ptr(topk_w),
                                 _ptr(logits), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)),
           "moe_router_topk")


def router_topk_limited(shape, x, Wg, allowed, topk_idx, topk_w, logits, ws, stream=None):
    _check(lib().moe_router_topk_limited(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(allowed), _ptr(topk_idx),
                                         _ptr(topk_w), _ptr(logits), _ptr(ws), ws.numel() if ws is not None else 0,
                                         _stream(stream)), "moe_router_topk_limited")


def expert_utilisation(shape, counts, utilisation, flags, stream=None):
    _check(lib().moe_expert_utilisation(ctypes.byref(shape), _ptr(counts), _ptr(utilisation), _ptr(flags),
                                        _stream(stream)), "moe_expert_utilisation")


def permute(shape, topk_idx, counts, offsets, perm_token, row_of, x, x_perm, ws, stream=None):
    _check(lib().moe_permute(ctypes.byref(shape), _ptr(topk_idx), _ptr(counts), _ptr(offsets), _ptr(perm_token),
                             _ptr(row_of), _ptr(x), _ptr(x_perm), _ptr(ws), ws.numel() if ws is not None else 0,
                             _stream(stream)), "moe_permute")


def grouped_swiglu(shape, x, x_perm, offsets, W1, W3, W2, s1, s3, s2, W1s, W3s, W2s, Y_perm, Y_shared, ws,
                   stream=None):
    _check(lib().moe_grouped_swiglu(ctypes.byref(shape), _ptr(x), _ptr(x_perm), _ptr(offsets), _ptr(W1), _ptr(W3),
                                    _ptr(W2), _ptr(s1), _ptr(s3), _ptr(s2), _ptr(W1s), _ptr(W3s), _ptr(W2s),
                                    _ptr(Y_perm), _ptr(Y_shared), _ptr(ws), ws.numel() if ws is not None else 0,
                                    _stream(stream)), "moe_grouped_swiglu")


def combine(shape, Y_perm, Y_shared, row_of, topk_w, y, stream=None):
    _check(lib().moe_combine(ctypes.byref(shape), _ptr(Y_perm), _ptr(Y_shared), _ptr(row_of), _ptr(topk_w), _ptr(y),
                             _stream(stream)), "moe_combine")


def combine_backward(shape, dy, Y_perm, row_of, topk_w, dO_perm, dw, stream=None):
    """Backward of the combine (moe_combine_backward): dO_perm rows and dw."""
    _check(lib().moe_combine_backward(ctypes.byref(shape), _ptr(dy), _ptr(Y_perm), _ptr(row_of), _ptr(topk_w),
                                      _ptr(dO_perm), _ptr(dw), _stream(stream)), "moe_combine_backward")


def router_backward(shape, logits, topk_idx, topk_w, dw, dlogits, stream=None):
    """Backward of the routing weights (moe_router_backward): dlogits [T, E]."""
    _check(lib().moe_router_backward(ctypes.byref(shape), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(dw),
                                     _ptr(dlogits), _stream(stream)), "moe_router_backward")


def forward(shape, x, Wg, bias, W1, W3, W2, s1, s3, s2, W1s, W3s, W2s, y, ws, topk_idx=None, topk_w=None,
            counts=None, stream=None):
    _check(lib().moe_forward(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3), _ptr(W2),
                             _ptr(s1), _ptr(s3), _ptr(s2), _ptr(W1s), _ptr(W3s), _ptr(W2s), _ptr(y), _ptr(topk_idx),
                             _ptr(topk_w), _ptr(counts), _ptr(ws), ws.numel() if ws is not None else 0,
                             _stream(stream)), "moe_forward")


def forward_launches(shape) -> int:
    """Kernel launches one moe_forward call issues for this shape on the current device."""
    n = int(lib().moe_forward_launches(ctypes.byref(shape)))
    if n < 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_forward_launches")
    return n


def forward_ep(shape, ep_rank, ep_size, x, Wg, bias, W1, W3, W2, s1, s3, s2, W1s, W3s, W2s, y, ws, topk_idx=None,
               topk_w=None, counts=None, stream=None):
    """This rank's share of the expert-parallel layer (moe_forward_ep): W1/W3/W2
    (and scales) hold the rank's E/ep_size experts, W1s/W3s/W2s its slice of
    the shared expert's hidden features; y receives the partial sum that
    all_reduce_partial (or any sum over ranks) completes."""
    _check(lib().moe_forward_ep(ctypes.byref(shape), int(ep_rank), int(ep_size), _ptr(x), _ptr(Wg), _ptr(bias),
                                _ptr(W1), _ptr(W3), _ptr(W2), _ptr(s1), _ptr(s3), _ptr(s2), _ptr(W1s), _ptr(W3s),
                                _ptr(W2s), _ptr(y), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(ws),
                                ws.numel() if ws is not None else 0, _stream(stream)), "moe_forward_ep")


def forward_profiled(shape, x, Wg, bias, W1, W3, W2, s1, s3, s2, W1s, W3s, W2s, y, ws, events, topk_idx=None,
                     topk_w=None, counts=None, stream=None):
    """forward() that also records `events` (NUM_STAGE_EVENTS torch.cuda.Event
    objects with timing enabled) at the stage boundaries."""
    if len(events) != NUM_STAGE_EVENTS:
        raise ValueError(f"need {NUM_STAGE_EVENTS} events")
    for ev in events:
        if not ev.cuda_event:  # torch creates the CUDA event on its first record
            ev.record()
    handles = (ctypes.c_void_p * NUM_STAGE_EVENTS)(*[ev.cuda_event for ev in events])
    _check(lib().moe_forward_profiled(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3),
                                      _ptr(W2), _ptr(s1), _ptr(s3), _ptr(s2), _ptr(W1s), _ptr(W3s), _ptr(W2s),
                                      _ptr(y), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(ws),
                                      ws.numel() if ws is not None else 0, _stream(stream), handles),
           "moe_forward_profiled")


def shared_expert(shape, x, W1s, W3s, W2s, Y_shared, ws, stream=None):
    """The shared expert alone (moe_shared_expert): Y_shared [T, d] fp32."""
    _check(lib().moe_shared_expert(ctypes.byref(shape), _ptr(x), _ptr(W1s), _ptr(W3s), _ptr(W2s), _ptr(Y_shared),
                                   _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)), "moe_shared_expert")


def ep_regroup_layout(n_src, E_local, recv_counts, offsets_local, to_expert_major, to_source_major, stream=None):
    """Expert-major order of rows received from n_src ranks (moe_ep_regroup_layout)."""
    _check(lib().moe_ep_regroup_layout(int(n_src), int(E_local), _ptr(recv_counts), _ptr(offsets_local),
                                       _ptr(to_expert_major), _ptr(to_source_major), _stream(stream)),
           "moe_ep_regroup_layout")


def gather_rows(src, index, dst, stream=None):
    """dst[r] = src[index[r]] for every row of dst (moe_gather_rows, bf16 rows)."""
    rows = int(dst.shape[0])
    if rows == 0:
        return
    _check(lib().moe_gather_rows(_ptr(src), _ptr(index), rows, int(dst.shape[1]), _ptr(dst), _stream(stream)),
           "moe_gather_rows")


def backward_workspace_size(shape: MoeShape) -> int:
    return int(lib().moe_backward_workspace_size(ctypes.byref(shape)))


def alloc_backward_workspace(shape: MoeShape, device="cuda") -> torch.Tensor:
    n = backward_workspace_size(shape)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_backward_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def backward(shape, x, Wg, bias, W1, W3, W2, W1s, W3s, W2s, dy, dx, dWg, dW1, dW3, dW2, dW1s, dW3s, dW2s, ws,
             stream=None):
    """Gradient of sum(dy * y) of the layer (moe_backward): dx, dWg, dW1, dW3,
    dW2 and the shared expert's dW1s, dW3s, dW2s, in shape.y_dtype."""
    _check(lib().moe_backward(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3), _ptr(W2),
                              _ptr(W1s), _ptr(W3s), _ptr(W2s), _ptr(dy), _ptr(dx), _ptr(dWg), _ptr(dW1), _ptr(dW3),
                              _ptr(dW2), _ptr(dW1s), _ptr(dW3s), _ptr(dW2s), _ptr(ws),
                              ws.numel() if ws is not None else 0, _stream(stream)), "moe_backward")


def forward_train(shape, x, Wg, bias, W1, W3, W2, W1s, W3s, W2s, y, ws, stream=None):
    """moe_forward_train: the layer's y, keeping the forward's state in the
    backward workspace `ws` for backward_saved."""
    _check(lib().moe_forward_train(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3), _ptr(W2),
                                   _ptr(W1s), _ptr(W3s), _ptr(W2s), _ptr(y), _ptr(ws),
                                   ws.numel() if ws is not None else 0, _stream(stream)), "moe_forward_train")


def backward_saved(shape, x, Wg, W1, W3, W2, W1s, W3s, W2s, dy, dx, dWg, dW1, dW3, dW2, dW1s, dW3s, dW2s, ws,
                   stream=None):
    """moe_backward_saved: every gradient from the state forward_train left in `ws`."""
    _check(lib().moe_backward_saved(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(W1s),
                                    _ptr(W3s), _ptr(W2s), _ptr(dy), _ptr(dx), _ptr(dWg), _ptr(dW1), _ptr(dW3),
                                    _ptr(dW2), _ptr(dW1s), _ptr(dW3s), _ptr(dW2s), _ptr(ws),
                                    ws.numel() if ws is not None else 0, _stream(stream)), "moe_backward_saved")


# ------------------------------------------------------------------ few tokens, MXFP4, gradients
# The calls below run on the device of their tensors, whichever is current, and
# by default on that device's current stream.
_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_DTYPES = {_F32: MOE_F32, _BF16: MOE_BF16}


def _on(device, stream, call):
    if device.type != "cuda":
        raise ValueError(f"libmoe works on CUDA tensors, got one on {device}")
    if stream is None:
        # the handle alone: a Stream object costs 2 us, a quarter of a small call
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        raise ValueError(f"stream on {stream.device} for tensors on {device}")
    else:
        raw = stream.cuda_stream
    if device.index == torch.cuda.current_device():
        return call(raw)
    with torch.cuda.device(device):
        return call(raw)


def _adr(t, device):
    """Address of a contiguous tensor on `device` (None stays None)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    if t.device != device:
        raise ValueError(f"tensors on {t.device} and {device} in one call")
    return t.data_ptr()


def _fit(t, device, n, dtype, what):
    """_adr of a tensor with at least n elements of a type (an int: of any type of so many bytes)."""
    if t is None:
        return None  # the library's to refuse
    if t.numel() < n or (t.dtype is not dtype and t.element_size() != dtype):
        kind = f"{dtype}-byte values" if isinstance(dtype, int) else dtype
        raise ValueError(f"{what} has {t.numel()} elements of {t.dtype}, {n} of {kind} needed")
    return _adr(t, device)


def _dtype(t):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"fp32 or bf16 tensors only, got {t.dtype}") from None


def _sized(t, n, what):
    if t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} elements, {n} needed")


def few_workspace_size(shape: MoeShape) -> int:
    return int(lib().moe_few_workspace_size(ctypes.byref(shape)))


def alloc_few_workspace(shape: MoeShape, device="cuda") -> torch.Tensor:
    n = few_workspace_size(shape)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_few_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def forward_few(shape, x, Wg, bias, W1, W3, W2, s1, s3, s2, W1s, W3s, W2s, y, ws, topk_idx=None, topk_w=None,
                counts=None, stream=None):
    """The layer for at most MOE_FEW_MAX_TOKENS tokens (moe_forward_few), bf16,
    e4m3 or MXFP4 experts; arguments as forward().  Tensors that are shorter than
    the shape needs, or of another type, are refused."""
    dev, kind = x.device, shape.w_dtype
    T, d, E, k, I, S = shape.T, shape.d, shape.E, shape.k, shape.inter, shape.shared_inter
    n = E * d * I  # values of a matrix; its codes and scales
    codes, wide, scales, per_scale = ((n, _BF16, 0, None) if kind == MOE_BF16 else
                                      (n, 1, n // 16384, _F32) if kind == MOE_E4M3 else (n // 2, 1, n // 32, 1))
    if not scales:
        s1 = s3 = s2 = None
    if not S:
        W1s = W3s = W2s = None
    if shape.route != MOE_ROUTE_SIGMOID_GROUP:
        bias = None
    a = (_fit(x, dev, T * d, _BF16, "x"), _fit(Wg, dev, E * d, _BF16, "Wg"), _fit(bias, dev, E, _F32, "bias"),
         _fit(W1, dev, codes, wide, "W1"), _fit(W3, dev, codes, wide, "W3"), _fit(W2, dev, codes, wide, "W2"),
         _fit(s1, dev, scales, per_scale, "s1"), _fit(s3, dev, scales, per_scale, "s3"),
         _fit(s2, dev, scales, per_scale, "s2"), _fit(W1s, dev, d * S, _BF16, "W1s"),
         _fit(W3s, dev, d * S, _BF16, "W3s"), _fit(W2s, dev, S * d, _BF16, "W2s"),
         _fit(y, dev, T * d, _F32 if shape.y_dtype == MOE_F32 else _BF16, "y"),
         _fit(topk_idx, dev, T * k, _I32, "topk_idx"), _fit(topk_w, dev, T * k, _F32, "topk_w"),
         _fit(counts, dev, E, _I32, "counts"), _adr(ws, dev))
    fn, size = lib().moe_forward_few, ws.numel()
    _check(_on(dev, stream, lambda st: fn(ctypes.byref(shape), *a, size, st)), "moe_forward_few")


def mx_quantise(src, codes, scales, up=None, stream=None):
    """MXFP4 codes and scale bytes of rows (moe_mx_quantise): src [..., cols]
    fp32 or bf16, innermost dimension contiguous and the rows evenly spaced;
    codes [..., cols/2] and scales [..., cols/32] uint8.  up: quantise
    silu(src) * up instead."""
    cols = src.shape[-1]
    rows = src.numel() // cols if cols else 0
    ld = _row_stride(src)
    if up is not None and (up.shape != src.shape or up.dtype != src.dtype or _row_stride(up) != ld):
        raise ValueError("src and up must have the same shape, type and strides")
    _sized(codes, rows * cols // 2, "codes")
    _sized(scales, rows * cols // 32, "scales")
    dev, dt = src.device, _dtype(src)
    c, s = _adr(codes, dev), _adr(scales, dev)
    u = None
    if up is not None:
        if up.device != dev:
            raise ValueError(f"tensors on {up.device} and {dev} in one call")
        u = up.data_ptr()
    fn = lib().moe_mx_quantise
    _check(_on(dev, stream, lambda st: fn(src.data_ptr(), u, dt, rows, cols, ld, c, s, st)), "moe_mx_quantise")


def _row_stride(t):
    """Elements between neighbouring rows of a tensor whose rows are evenly spaced."""
    if t.dim() > 0 and t.is_contiguous():
        return t.shape[-1]
    if t.dim() == 0 or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("rows must be contiguous")
    if t.dim() == 2:
        ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
        if ld >= t.shape[1]:
            return ld
    raise ValueError("rows must be evenly spaced and must not overlap")


def mx_quantise_weights(W, codes, scales, stream=None):
    """MXFP4 codes [E, N, K/2] and scale bytes [E, N, K/32] of weights [E, K, N]
    (moe_mx_quantise_weights); a matrix [K, N] is one expert."""
    if W.dim() not in (2, 3):
        raise ValueError("weights are [E, K, N] or [K, N]")
    E, (K, N) = (W.shape[0] if W.dim() == 3 else 1), W.shape[-2:]
    _sized(codes, E * N * K // 2, "codes")
    _sized(scales, E * N * K // 32, "scales")
    dev, dt = W.device, _dtype(W)
    w, c, s = _adr(W, dev), _adr(codes, dev), _adr(scales, dev)
    fn = lib().moe_mx_quantise_weights
    _check(_on(dev, stream, lambda st: fn(w, dt, E, K, N, c, s, st)), "moe_mx_quantise_weights")


def mx_dequantise(codes, scales, dst, stream=None):
    """The values of MXFP4 codes (moe_mx_dequantise) in dst [..., cols], fp32 or bf16."""
    cols = dst.shape[-1]
    rows = dst.numel() // cols if cols else 0
    _sized(codes, rows * cols // 2, "codes")
    _sized(scales, rows * cols // 32, "scales")
    dev, dt = dst.device, _dtype(dst)
    c, s, d = _adr(codes, dev), _adr(scales, dev), _adr(dst, dev)
    fn = lib().moe_mx_dequantise
    _check(_on(dev, stream, lambda st: fn(c, s, rows, cols, d, dt, st)), "moe_mx_dequantise")


def alloc_mx_product_workspace(rows: int, E: int, device="cuda") -> torch.Tensor:
    n = int(lib().moe_mx_product_workspace_size(int(rows), int(E)))
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_mx_product_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def mx_grouped_product(A, A_scales, offsets, W, W_scales, Y, ws, stream=None):
    """Y[r] = A[r] W[e]^T for the rows of each expert (moe_mx_grouped_product):
    A codes [rows, K/2], scales [rows, K/32]; offsets [E + 1] int32; W codes
    [E, N, K/2], scales [E, N, K/32]; Y [rows, N] fp32 or bf16."""
    rows, K = A.shape[0], 2 * A.shape[1]
    E, N = W.shape[0], W.shape[1]
    if W.shape[2] * 2 != K or Y.shape != (rows, N) or offsets.dtype != torch.int32:
        raise ValueError("shapes of A, W, Y or the type of offsets do not fit together")
    _sized(offsets, E + 1, "offsets")
    _sized(A_scales, rows * K // 32, "A_scales")
    _sized(W_scales, E * N * K // 32, "W_scales")
    dev, dt = A.device, _dtype(Y)
    a = [_adr(t, dev) for t in (A, A_scales, offsets, W, W_scales, Y)]
    w, size = _adr(ws, dev), ws.numel()
    fn = lib().moe_mx_grouped_product
    _check(_on(dev, stream, lambda st: fn(rows, E, K, N, *a, dt, w, size, st)), "moe_mx_grouped_product")


def alloc_grad_workspace(n: int, device="cuda") -> torch.Tensor:
    size = int(lib().moe_grad_workspace_size(int(n)))
    if size == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_grad_workspace_size")
    return torch.empty(size, dtype=torch.uint8, device=device)


def _tensor_list(grads, out, device):
    arr = (MoeTensor * max(1, len(grads)))()
    if out is not None and len(out) != len(grads):
        raise ValueError(f"{len(out)} outputs for {len(grads)} tensors")
    for i, g in enumerate(grads):
        o = None
        if out is not None:
            if out[i].dtype != g.dtype or out[i].shape != g.shape:
                raise ValueError("an output differs from its tensor in type or shape")
            o = _adr(out[i], device)
        arr[i] = (_adr(g, device), o, g.numel(), _dtype(g))
    return arr


def grad_norm(grads, norm, ws, stream=None):
    """norm [1] fp32 = the global norm of the tensors of `grads` (moe_grad_norm)."""
    dev = norm.device
    arr, n = _tensor_list(grads, None, dev), len(grads)
    o, w, size = _fit(norm, dev, 1, _F32, "norm"), _adr(ws, dev), ws.numel()
    fn = lib().moe_grad_norm
    _check(_on(dev, stream, lambda st: fn(arr, n, o, w, size, st)), "moe_grad_norm")


def grad_clip(grads, max_norm, norm, ws, out=None, stream=None):
    """Scale the tensors of `grads` by min(1, max_norm / (norm + 1e-6)) of their
    global norm (moe_grad_clip), in place or into the tensors of `out`; norm [1]
    fp32 receives the norm before clipping (None: not returned)."""
    dev = ws.device
    arr, n = _tensor_list(grads, out, dev), len(grads)
    o, w, size = _fit(norm, dev, 1, _F32, "norm"), _adr(ws, dev), ws.numel()
    fn = lib().moe_grad_clip
    _check(_on(dev, stream, lambda st: fn(arr, n, max_norm, o, w, size, st)), "moe_grad_clip")


def check_device_status(ws, stream=None) -> tuple[int, int]:
    raw = ctypes.c_uint32(0)
    rc = lib().moe_check_device_status(_ptr(ws), _stream(stream), ctypes.byref(raw))
    return rc, raw.value


def version() -> str:
    return lib().moe_version().decode()
