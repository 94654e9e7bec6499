"""ctypes binding of libmoe (include/moe.h): argument marshalling only.

Each function has the C entry point's name and takes torch tensors (device
memory) in place of pointers. Every step of the layer runs in libmoe's CUDA
kernels; this module computes nothing. If libmoe.so has not been built the
import fails loudly: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_TIMEOUT = range(6)
MOE_F32, MOE_BF16 = 0, 1

# Every symbol include/moe.h declares.
EXPORTED = (
    "moe_workspace_size", "moe_router_topk", "moe_topk_from_logits", "moe_topk_from_logits_noisy",
    "moe_dispatch", "moe_layer_forward_noisy",
    "moe_grouped_ffn", "moe_combine", "moe_layer_forward", "moe_layer_forward_profiled",
    "moe_expert_stats", "moe_bias_update",
    "moe_check_status", "moe_status_string", "moe_kernel_launch_count", "moe_dispatch_noalloc",
    "moe_expert_gemms", "moe_gather_rows", "moe_ep_local_order",
    "moe_route", "moe_route_backward", "moe_layer_forward_routed", "moe_combine_backward",
    "moe_norm_workspace_size", "moe_block_norm", "moe_block_norm_backward",
    "moe_linear_workspace_size", "moe_linear", "moe_linear_backward",
)

# Named choices of the block operators' descriptors, in the header's order.
SCORES = ("softmax", "sigmoid")
GATES = ("none", "channel", "token", "full")
ACTS = ("none", "gelu", "silu")


class MoELayerDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "E", "K", "D", "Ds", "dtype", "cf_num", "cf_den")]


class MoELayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_router", "w1", "w2", "ws1", "ws2", "expert_bias")]


class MoERouting(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_idx", "topk_w", "counts", "offsets", "perm", "inv", "logits")]


class MoEStats(ctypes.Structure):
    _fields_ = [("num_copies", ctypes.c_int64), ("overflow", ctypes.c_int64),
                ("capacity", ctypes.c_int32), ("max_load", ctypes.c_int32),
                ("min_load", ctypes.c_int32), ("num_stragglers", ctypes.c_int32),
                ("skew_ratio", ctypes.c_double), ("gini", ctypes.c_double),
                ("overflow_rate", ctypes.c_double), ("max_over_mean", ctypes.c_double)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class MoERouteDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "E", "K", "score", "groups", "topk_groups", "group_top",
                                              "renorm")] + [("scale", ctypes.c_float)]


class MoENormDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "dtype", "gate")] + \
               [("eps", ctypes.c_float), ("alpha", ctypes.c_float)]


class MoELinearDesc(ctypes.Structure):
    # the header's `in` and `out`
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "n_in", "n_out", "dtype", "act")]


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libmoe.so is not built ({LIB_PATH}); run `python -m fine_grained_moe_router_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, S = ctypes.c_void_p, ctypes.c_size_t
    D = ctypes.POINTER(MoELayerDesc)
    sig = {
        "moe_workspace_size": (S, [D]),
        "moe_router_topk": (ctypes.c_int, [D, P, P, P, P, P, P, P, S, P]),
        "moe_topk_from_logits": (ctypes.c_int, [D, P, P, P, P, P]),
        "moe_topk_from_logits_noisy": (ctypes.c_int, [D, P, P, P, P, P, P]),
        "moe_layer_forward_noisy": (ctypes.c_int, [D, ctypes.POINTER(MoELayerWeights), P, P, P,
                                                   ctypes.POINTER(MoERouting), P, S, P]),
        "moe_dispatch": (ctypes.c_int, [D, P, P, P, P, P, P, S, P]),
        "moe_grouped_ffn": (ctypes.c_int, [D, P, P, P, P, P, P, P, P, P, P, S, P]),
        "moe_combine": (ctypes.c_int, [D, P, P, P, P, P, P]),
        "moe_layer_forward": (ctypes.c_int, [D, ctypes.POINTER(MoELayerWeights), P, P,
                                             ctypes.POINTER(MoERouting), P, S, P]),
        "moe_layer_forward_profiled": (ctypes.c_int, [D, ctypes.POINTER(MoELayerWeights), P, P,
                                                      ctypes.POINTER(MoERouting), P, S, P,
                                                      ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]),
        "moe_expert_stats": (ctypes.c_int, [D, P, P, ctypes.POINTER(MoEStats), P, S, P]),
        "moe_bias_update": (ctypes.c_int, [D, P, P, ctypes.c_float, P]),
        "moe_check_status": (ctypes.c_int, [P, S, P]),
        "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_kernel_launch_count": (ctypes.c_uint64, []),
        "moe_dispatch_noalloc": (ctypes.c_int, [D, P, P, P, P, P, P]),
        "moe_expert_gemms": (ctypes.c_int, [D, ctypes.POINTER(MoELayerWeights), P, P, S, P]),
        "moe_gather_rows": (ctypes.c_int, [P, ctypes.c_int64, P, ctypes.c_int32, ctypes.c_int64,
                                           ctypes.c_int64, P, P]),
        "moe_ep_local_order": (ctypes.c_int, [P, ctypes.c_int32, ctypes.c_int32, P, P, P,
                                              ctypes.c_int64, P]),
        "moe_route": (ctypes.c_int, [P, P, P, P, P, P]),
        "moe_route_backward": (ctypes.c_int, [P, P, P, P, P, P]),
        "moe_layer_forward_routed": (ctypes.c_int, [D, P, ctypes.POINTER(MoELayerWeights), P, P,
                                                    ctypes.POINTER(MoERouting), P, S, P]),
        "moe_combine_backward": (ctypes.c_int, [D, P, P, P, P, P, P, P]),
        "moe_norm_workspace_size": (S, [P]),
        "moe_block_norm": (ctypes.c_int, [P] * 9),
        "moe_block_norm_backward": (ctypes.c_int, [P] * 14 + [S, P]),
        "moe_linear_workspace_size": (S, [P]),
        "moe_linear": (ctypes.c_int, [P] * 8 + [S, P]),
        "moe_linear_backward": (ctypes.c_int, [P] * 9 + [S, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.moe_status_string(int(status)).decode()


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where)


def make_desc(T: int, H: int, E: int, K: int, D: int, Ds: int = 0, dtype: int = MOE_BF16,
              cf: tuple = (5, 4)) -> MoELayerDesc:
    return MoELayerDesc(T, H, E, K, D, Ds, dtype, cf[0], cf[1])


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return MOE_BF16
    if dt == torch.float32:
        return MOE_F32
    raise ValueError(f"unsupported layer dtype {dt}")


def moe_workspace_size(desc: MoELayerDesc) -> int:
    return int(lib.moe_workspace_size(ctypes.byref(desc)))


def alloc_workspace(desc, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for a layer, norm or linear descriptor."""
    size = moe_norm_workspace_size if isinstance(desc, MoENormDesc) else \
        moe_linear_workspace_size if isinstance(desc, MoELinearDesc) else moe_workspace_size
    n = size(desc)
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, size.__name__)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_router_topk(desc, x, w_router, bias, logits, topk_idx, topk_w, ws, stream=None):
    _check(lib.moe_router_topk(ctypes.byref(desc), _p(x), _p(w_router), _p(bias), _p(logits),
                               _p(topk_idx), _p(topk_w), _p(ws), ws.numel() if ws is not None else 0,
                               _stream(stream)), "moe_router_topk")


def moe_topk_from_logits(desc, logits, bias, topk_idx, topk_w, stream=None):
    _check(lib.moe_topk_from_logits(ctypes.byref(desc), _p(logits), _p(bias), _p(topk_idx),
                                    _p(topk_w), _stream(stream)), "moe_topk_from_logits")


def moe_topk_from_logits_noisy(desc, logits, bias, gumbel_noise, topk_idx, topk_w, stream=None):
    """Selection on (logits + bias) + gumbel_noise [T, E] fp32 (noisy routing)."""
    _check(lib.moe_topk_from_logits_noisy(ctypes.byref(desc), _p(logits), _p(bias),
                                          _p(gumbel_noise), _p(topk_idx), _p(topk_w),
                                          _stream(stream)), "moe_topk_from_logits_noisy")


def moe_dispatch(desc, topk_idx, counts, offsets, perm, inv, ws, stream=None):
    _check(lib.moe_dispatch(ctypes.byref(desc), _p(topk_idx), _p(counts), _p(offsets), _p(perm),
                            _p(inv), _p(ws), ws.numel() if ws is not None else 0, _stream(stream)),
           "moe_dispatch")


def moe_dispatch_noalloc(desc, topk_idx, counts, offsets, perm, inv, stream=None):
    """moe_dispatch without a workspace, for callers that cannot allocate device
    memory: its scratch is a fixed array inside libmoe (T*K <= 65536). Calls that
    overlap on the GPU share that array and race."""
    _check(lib.moe_dispatch_noalloc(ctypes.byref(desc), _p(topk_idx), _p(counts), _p(offsets),
                                    _p(perm), _p(inv), _stream(stream)), "moe_dispatch_noalloc")


def moe_grouped_ffn(desc, x, perm, offsets, w1, w2, ws1, ws2, y_rows, y_shared, ws, stream=None):
    _check(lib.moe_grouped_ffn(ctypes.byref(desc), _p(x), _p(perm), _p(offsets), _p(w1), _p(w2),
                               _p(ws1), _p(ws2), _p(y_rows), _p(y_shared), _p(ws),
                               ws.numel() if ws is not None else 0, _stream(stream)),
           "moe_grouped_ffn")


def moe_combine(desc, y_rows, topk_w, inv, y_shared, y, stream=None):
    _check(lib.moe_combine(ctypes.byref(desc), _p(y_rows), _p(topk_w), _p(inv), _p(y_shared),
                           _p(y), _stream(stream)), "moe_combine")


def make_weights(w_router, w1, w2, ws1=None, ws2=None, bias=None) -> MoELayerWeights:
    return MoELayerWeights(*(t.data_ptr() if t is not None else None
                             for t in (w_router, w1, w2, ws1, ws2, bias)))


def make_routing(topk_idx=None, topk_w=None, counts=None, offsets=None, perm=None, inv=None,
                 logits=None) -> MoERouting:
    return MoERouting(*(t.data_ptr() if t is not None else None
                        for t in (topk_idx, topk_w, counts, offsets, perm, inv, logits)))


def moe_layer_forward(desc, weights: MoELayerWeights, x, y, routing: Optional[MoERouting], ws,
                      stream=None):
    _check(lib.moe_layer_forward(ctypes.byref(desc), ctypes.byref(weights), _p(x), _p(y),
                                 ctypes.byref(routing) if routing is not None else None, _p(ws),
                                 ws.numel() if ws is not None else 0, _stream(stream)),
           "moe_layer_forward")


def moe_layer_forward_noisy(desc, weights: MoELayerWeights, x, gumbel_noise, y,
                            routing: Optional[MoERouting], ws, stream=None):
    """moe_layer_forward with Gumbel noise [T, E] fp32 added to the selection scores."""
    _check(lib.moe_layer_forward_noisy(ctypes.byref(desc), ctypes.byref(weights), _p(x),
                                       _p(gumbel_noise), _p(y),
                                       ctypes.byref(routing) if routing is not None else None,
                                       _p(ws), ws.numel() if ws is not None else 0,
                                       _stream(stream)), "moe_layer_forward_noisy")


FORWARD_STAGES = ("router", "dispatch", "gemm1", "gemm2", "combine")


def moe_layer_forward_profiled(desc, weights: MoELayerWeights, x, y, routing: Optional[MoERouting],
                               ws, events, stream=None):
    """moe_layer_forward recording torch.cuda.Event objects (6, timing-enabled)
    between its stages on the launching stream."""
    for e in events:                 # torch creates the CUDA event on its first record
        if not e.cuda_event:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib.moe_layer_forward_profiled(ctypes.byref(desc), ctypes.byref(weights), _p(x), _p(y),
                                          ctypes.byref(routing) if routing is not None else None,
                                          _p(ws), ws.numel() if ws is not None else 0,
                                          _stream(stream), arr, len(events)),
           "moe_layer_forward_profiled")


def moe_expert_gemms(desc, weights: MoELayerWeights, x, ws, stream=None) -> None:
    """The expert-GEMM launches of the last moe_layer_forward on `ws` again (timing)."""
    _check(lib.moe_expert_gemms(ctypes.byref(desc), ctypes.byref(weights), _p(x), _p(ws),
                                ws.numel() if ws is not None else 0, _stream(stream)),
           "moe_expert_gemms")


def moe_gather_rows(src, idx, divisor: int, dst, stream=None) -> None:
    """dst[r] = src[idx[r] // divisor] for every row of dst (row-major 2-D tensors)."""
    row_bytes = dst[0].numel() * dst.element_size() if dst.shape[0] else 16
    _check(lib.moe_gather_rows(_p(src), src.shape[0], _p(idx), int(divisor), dst.shape[0],
                               row_bytes, _p(dst), _stream(stream)), "moe_gather_rows")


def moe_ep_local_order(recv_counts, offsets, perm, inv, stream=None) -> None:
    """Expert-major order of the rows received from G ranks (recv_counts [G, El] int32)."""
    G, El = recv_counts.shape
    _check(lib.moe_ep_local_order(_p(recv_counts), G, El, _p(offsets),
                                  _p(perm) if perm.numel() else None,
                                  _p(inv) if inv.numel() else None, perm.numel(),
                                  _stream(stream)), "moe_ep_local_order")


def moe_expert_stats(desc, counts, straggler_mask, ws, stream=None) -> dict:
    out = MoEStats()
    _check(lib.moe_expert_stats(ctypes.byref(desc), _p(counts), _p(straggler_mask),
                                ctypes.byref(out), _p(ws), ws.numel() if ws is not None else 0,
                                _stream(stream)), "moe_expert_stats")
    return out.as_dict()


def moe_bias_update(desc, counts, bias, gamma: float, stream=None) -> None:
    """Updates `bias` [E] fp32 in place from the accumulated `counts` [E] int32."""
    _check(lib.moe_bias_update(ctypes.byref(desc), _p(counts), _p(bias), ctypes.c_float(gamma),
                               _stream(stream)), "moe_bias_update")


def moe_kernel_launch_count() -> int:
    return int(lib.moe_kernel_launch_count())


def moe_check_status(ws, stream=None) -> int:
    return int(lib.moe_check_status(_p(ws), ws.numel(), _stream(stream)))


# ---------------------------------------------------------------------------
# Block operators: routing with groups, combine gradient, block norms, linear
# layer. Beside the library's own checks, these check each tensor's type, shape
# and layout, which the C ABI cannot see.
# ---------------------------------------------------------------------------
_TORCH = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def _arg(name, t, shape, dtype, device=None, optional=False):
    """Address of a contiguous tensor of this shape and type, on CUDA device number
    `device` if given; 0 for None where that is allowed."""
    if t is None:
        if optional:
            return 0
        raise ValueError(f"{name} is missing")
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and \
            (device is None or t.get_device() == device):
        return t.data_ptr()
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    raise ValueError(f"{name} is on {t.device}, the other tensors are on device {device}")


def _space(ws, device):
    """Address and length of a workspace on CUDA device number `device`. The kernels write
    to it: one on the host, or one that repeats its bytes, is not a workspace."""
    if ws is None:
        raise ValueError("ws is missing")
    if ws.get_device() != device:
        raise ValueError(f"ws is on {ws.device}, the other tensors are on device {device}")
    if not ws.is_contiguous():
        raise ValueError("ws is not contiguous")
    return ws.data_ptr(), ws.numel()


def _place(t, stream):
    """The device number of `t`, and the stream to launch on. A library call launches on
    the current device, so that has to be the tensors' own."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"the tensors are on {t.device}, not on a CUDA device")
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {t.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    return dev, stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _choice(names, name, what):
    try:
        return names.index(name)
    except ValueError:
        raise ValueError(f"{what}: expected one of {', '.join(names)}, got {name!r}") from None


def make_route(T: int, E: int, K: int, score: str = "sigmoid", groups: int = 1, topk_groups: int = 1,
               group_top: int = 1, renorm: bool = True, scale: float = 1.0) -> MoERouteDesc:
    """Descriptor of moe_route: `score` "softmax" or "sigmoid"; `groups` equal
    groups of experts of which the `topk_groups` best are kept, each worth the sum
    of its `group_top` best choices; weights renormalised and scaled."""
    return MoERouteDesc(T, E, K, _choice(SCORES, score, "score"), groups, topk_groups, group_top,
                        int(bool(renorm)), scale)


def moe_route(desc: MoERouteDesc, logits, bias, topk_idx, topk_w, stream=None) -> None:
    """Fills topk_idx [T, K] int32 and topk_w [T, K] fp32 from logits [T, E] fp32;
    the bias [E] fp32 (or None) takes part in the choice only."""
    dev, st = _place(logits, stream)
    f32, row, out = torch.float32, (desc.T, desc.E), (desc.T, desc.K)
    _check(lib.moe_route(ctypes.addressof(desc), _arg("logits", logits, row, f32),
                         _arg("bias", bias, (desc.E,), f32, dev, True),
                         _arg("topk_idx", topk_idx, out, torch.int32, dev),
                         _arg("topk_w", topk_w, out, f32, dev), st), "moe_route")


def moe_route_backward(desc: MoERouteDesc, logits, topk_idx, d_topk_w, d_logits, stream=None) -> None:
    """d_logits [T, E] fp32 from d_topk_w [T, K] fp32, the choice held fixed."""
    dev, st = _place(logits, stream)
    f32, row, out = torch.float32, (desc.T, desc.E), (desc.T, desc.K)
    _check(lib.moe_route_backward(ctypes.addressof(desc), _arg("logits", logits, row, f32),
                                  _arg("topk_idx", topk_idx, out, torch.int32, dev),
                                  _arg("d_topk_w", d_topk_w, out, f32, dev),
                                  _arg("d_logits", d_logits, row, f32, dev), st),
           "moe_route_backward")


def moe_layer_forward_routed(desc, route: MoERouteDesc, weights: MoELayerWeights, x, y,
                             routing: Optional[MoERouting], ws, stream=None) -> None:
    """moe_layer_forward with the routing of moe_route (weights.expert_bias is its bias)."""
    dev, st = _place(x, stream)
    dt = _TORCH[desc.dtype]
    _check(lib.moe_layer_forward_routed(ctypes.byref(desc), ctypes.addressof(route),
                                        ctypes.byref(weights),
                                        _arg("x", x, (desc.T, desc.H), dt),
                                        _arg("y", y, (desc.T, desc.H), dt, dev),
                                        ctypes.byref(routing) if routing is not None else None,
                                        *(_space(ws, dev) if ws is not None else (None, 0)), st),
           "moe_layer_forward_routed")


def moe_combine_backward(desc, dy, y_rows, topk_w, inv, d_y_rows, d_topk_w, stream=None) -> None:
    """Gradient of moe_combine: d_y_rows [T*K, H] (layer dtype) and d_topk_w [T, K] fp32."""
    dev, st = _place(dy, stream)
    T, H, K, dt = desc.T, desc.H, desc.K, _TORCH[desc.dtype]
    if inv.numel() != T * K:
        raise ValueError(f"inv: expected {T * K} entries, got {tuple(inv.shape)}")
    _check(lib.moe_combine_backward(ctypes.byref(desc), _arg("dy", dy, (T, H), dt),
                                    _arg("y_rows", y_rows, (T * K, H), torch.float32, dev),
                                    _arg("topk_w", topk_w, (T, K), torch.float32, dev),
                                    _arg("inv", inv, tuple(inv.shape), torch.int32, dev),
                                    _arg("d_y_rows", d_y_rows, (T * K, H), dt, dev),
                                    _arg("d_topk_w", d_topk_w, (T, K), torch.float32, dev), st),
           "moe_combine_backward")


def make_norm(T: int, H: int, dtype: int = MOE_BF16, gate: str = "none", alpha: float = 1.0,
              eps: float = 1e-6) -> MoENormDesc:
    """Descriptor of moe_block_norm: `gate` "none", "channel" [H], "token" [T] or
    "full" [T, H]; `alpha` scales the block's contribution."""
    return MoENormDesc(T, H, dtype, _choice(GATES, gate, "gate"), eps, alpha)


def moe_norm_workspace_size(desc: MoENormDesc) -> int:
    return int(lib.moe_norm_workspace_size(ctypes.addressof(desc)))


def _gate_shape(desc):
    return (None, (desc.H,), (desc.T,), (desc.T, desc.H))[desc.gate]


def moe_block_norm(desc: MoENormDesc, h, y=None, w_post=None, gate=None, w_pre=None, h_out=None,
                   x=None, stream=None) -> None:
    """h_out = h + alpha * gate * u with u = y, or rms(y) * w_post; x = rms(h_out) * w_pre.
    Without y: x = rms(h) * w_pre."""
    dev, st = _place(h, stream)
    row, col, dt = (desc.T, desc.H), (desc.H,), _TORCH[desc.dtype]
    _check(lib.moe_block_norm(ctypes.addressof(desc), _arg("h", h, row, dt),
                              _arg("y", y, row, dt, dev, True),
                              _arg("w_post", w_post, col, dt, dev, True),
                              _arg("gate", gate, _gate_shape(desc), dt, dev, True),
                              _arg("w_pre", w_pre, col, dt, dev, True),
                              _arg("h_out", h_out, row, dt, dev, True),
                              _arg("x", x, row, dt, dev, True), st), "moe_block_norm")


def moe_block_norm_backward(desc: MoENormDesc, d_h_out, d_x, h_out, y, w_post, gate, w_pre, d_h,
                            d_y, d_w_post, d_gate, d_w_pre, ws, stream=None) -> None:
    """Gradients of moe_block_norm; None leaves an input or output out. The weights'
    and the channel and token gates' gradients are fp32, the others of the layer dtype."""
    dev, st = _place(ws, stream)
    row, col, dt, f32 = (desc.T, desc.H), (desc.H,), _TORCH[desc.dtype], torch.float32
    shape = _gate_shape(desc)
    g_dt = dt if shape == row and desc.gate == 3 else f32
    _check(lib.moe_block_norm_backward(
        ctypes.addressof(desc), _arg("d_h_out", d_h_out, row, dt, dev, True),
        _arg("d_x", d_x, row, dt, dev, True), _arg("h_out", h_out, row, dt, dev, True),
        _arg("y", y, row, dt, dev, True), _arg("w_post", w_post, col, dt, dev, True),
        _arg("gate", gate, shape, dt, dev, True), _arg("w_pre", w_pre, col, dt, dev, True),
        _arg("d_h", d_h, row, dt, dev, True), _arg("d_y", d_y, row, dt, dev, True),
        _arg("d_w_post", d_w_post, col, f32, dev, True),
        _arg("d_gate", d_gate, shape, g_dt, dev, True),
        _arg("d_w_pre", d_w_pre, col, f32, dev, True), *_space(ws, dev), st),
        "moe_block_norm_backward")


def make_linear(T: int, n_in: int, n_out: int, dtype: int = MOE_BF16, act: str = "none") -> MoELinearDesc:
    """Descriptor of moe_linear: y = act(x W^T + bias) + residual; `act` "none",
    "gelu" (erf form) or "silu"."""
    return MoELinearDesc(T, n_in, n_out, dtype, _choice(ACTS, act, "act"))


MOE_LINEAR_WS_HEAD = 2048   # the header's: bytes of a linear workspace that have to be zero


def moe_linear_workspace_size(desc: MoELinearDesc) -> int:
    return int(lib.moe_linear_workspace_size(ctypes.addressof(desc)))


def moe_linear(desc: MoELinearDesc, x, w, bias, residual, pre, y, ws, stream=None) -> None:
    """y [T, out] = act(x w^T + bias) + residual; bias, residual and pre (which receives
    the activation's input) may be None."""
    dev, st = _place(x, stream)
    dt, out = _TORCH[desc.dtype], (desc.T, desc.n_out)
    _check(lib.moe_linear(ctypes.addressof(desc), _arg("x", x, (desc.T, desc.n_in), dt),
                          _arg("w", w, (desc.n_out, desc.n_in), dt, dev),
                          _arg("bias", bias, (desc.n_out,), dt, dev, True),
                          _arg("residual", residual, out, dt, dev, True),
                          _arg("pre", pre, out, dt, dev, True), _arg("y", y, out, dt, dev),
                          *_space(ws, dev), st), "moe_linear")


def moe_linear_backward(desc: MoELinearDesc, dy, x, w, pre, dx, dw, d_bias, ws, stream=None) -> None:
    """Gradients of moe_linear: dx [T, in], dw [out, in] (layer dtype), d_bias [out] fp32;
    None leaves one out."""
    dev, st = _place(dy, stream)
    dt, out = _TORCH[desc.dtype], (desc.T, desc.n_out)
    _check(lib.moe_linear_backward(
        ctypes.addressof(desc), _arg("dy", dy, out, dt), _arg("x", x, (desc.T, desc.n_in), dt, dev, True),
        _arg("w", w, (desc.n_out, desc.n_in), dt, dev, True), _arg("pre", pre, out, dt, dev, True),
        _arg("dx", dx, (desc.T, desc.n_in), dt, dev, True),
        _arg("dw", dw, (desc.n_out, desc.n_in), dt, dev, True),
        _arg("d_bias", d_bias, (desc.n_out,), torch.float32, dev, True), *_space(ws, dev), st),
        "moe_linear_backward")
