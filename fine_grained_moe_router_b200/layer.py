"""Layers with device-resident weights: thin convenience wrappers over the C ABI.

``MoELayer`` keeps the weights and a workspace of one fine-grained MoE FFN
layer and calls ``moe_layer_forward`` / ``moe_expert_stats``; ``MoEBlock`` puts
the norms and the residual around it (``moe_block_norm``); ``DenseFFN`` is a
dense two-layer feed-forward with its gradients (``moe_linear``).
"""
from __future__ import annotations

import contextlib
import threading
from typing import Optional

import torch

from . import _binding as B


# The launches of one call follow one another on their stream: calls of other threads on
# the same stream, and so with the same workspace, do not come between them.
_launching = threading.Lock()


def _on(stream):
    """Context in which tensors are allocated for use on `stream` (a torch stream or a
    raw handle; None: the current one). A temporary that is dropped while its kernels
    still run is then only reused behind them."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


class MoELayer:
    """Forward pass of one fine-grained MoE layer (router, dispatch, grouped
    expert FFN with an optional shared expert, combine) on one GPU.

    Weights (device tensors, nn.Linear [out, in] layout): w_router [E, H],
    w1 [E, D, H], w2 [E, H, D], optional shared expert ws1 [Ds, H] and
    ws2 [H, Ds], optional fp32 expert bias [E]. All weight tensors share one
    dtype (torch.float32 or torch.bfloat16).

    `route`: None for the layer's own softmax(l + B) routing, or the choices of
    ``make_route`` (score, groups, topk_groups, group_top, renorm, scale) as a dict
    for routing with a choice-only bias.

    The layer keeps one workspace: its calls, and those of a block around it, run one after
    the other, not on two streams at once. A captured graph uses it too, and stays valid
    until a larger batch makes the layer take a larger one."""

    def __init__(self, w_router, w1, w2, top_k: int, ws1=None, ws2=None, bias=None,
                 capacity_factor=(5, 4), route: Optional[dict] = None):
        self.E, self.H = w_router.shape
        self.D = w1.shape[1]
        self.Ds = 0 if ws1 is None else ws1.shape[0]
        self.K = int(top_k)
        self.dtype = w_router.dtype
        self.device = w_router.device
        self.cf = capacity_factor
        self.tensors = [t.contiguous() if t is not None else None
                        for t in (w_router, w1, w2, ws1, ws2, bias)]
        self.weights = B.make_weights(*self.tensors)
        self.route = dict(route) if route is not None else None
        self._ws: Optional[torch.Tensor] = None

    def route_desc(self, T: int) -> B.MoERouteDesc:
        return B.make_route(T, self.E, self.K, **(self.route or {}))

    def desc(self, T: int) -> B.MoELayerDesc:
        return B.make_desc(T, self.H, self.E, self.K, self.D, self.Ds, B.dtype_code(self.dtype),
                           self.cf)

    def workspace(self, T: int) -> torch.Tensor:
        need = B.moe_workspace_size(self.desc(T))
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
        return self._ws

    def routing_buffers(self, T: int) -> dict:
        dev, K, E = self.device, self.K, self.E
        i32 = torch.int32
        return {
            "topk_idx": torch.empty((T, K), dtype=i32, device=dev),
            "topk_w": torch.empty((T, K), dtype=torch.float32, device=dev),
            "counts": torch.empty(E, dtype=i32, device=dev),
            "offsets": torch.empty(E + 1, dtype=i32, device=dev),
            "perm": torch.empty(T * K, dtype=i32, device=dev),
            "inv": torch.empty(T * K, dtype=i32, device=dev),
            "logits": torch.empty((T, E), dtype=torch.float32, device=dev),
        }

    def forward(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, routing: Optional[dict] = None,
                stream=None, gumbel_noise: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y = MoE(x) for x [T, H]; fills `routing` (see routing_buffers) if given.
        gumbel_noise [T, E] fp32: noisy routing (Gumbel draws added to l + B)."""
        T = x.shape[0]
        if y is None:
            y = torch.empty_like(x)
        r = B.make_routing(**routing) if routing is not None else None
        if self.route is not None:
            if gumbel_noise is not None:
                raise ValueError("noisy routing belongs to the layer's own routing (route=None)")
            B.moe_layer_forward_routed(self.desc(T), self.route_desc(T), self.weights, x, y, r,
                                       self.workspace(T), stream)
        elif gumbel_noise is None:
            B.moe_layer_forward(self.desc(T), self.weights, x, y, r, self.workspace(T), stream)
        else:
            B.moe_layer_forward_noisy(self.desc(T), self.weights, x, gumbel_noise, y, r,
                                      self.workspace(T), stream)
        return y

    __call__ = forward

    def router_backward(self, dy: torch.Tensor, y_rows: torch.Tensor, routing: dict, stream=None) -> dict:
        """Gradients of the combine and of the routing weights, for a layer with `route`:
        from dy [T, H], the expert outputs y_rows [T*K, H] fp32 (moe_grouped_ffn) and the
        forward's routing. Returns d_y_rows [T*K, H] (layer dtype; the gradient that
        enters the experts), d_topk_w [T, K] and d_logits [T, E] fp32."""
        if self.route is None:
            raise ValueError("the routing gradient belongs to a layer with a route")
        T = dy.shape[0]
        with _on(stream):
            d_rows = torch.empty((T * self.K, self.H), dtype=self.dtype, device=self.device)
            d_w = torch.empty((T, self.K), dtype=torch.float32, device=self.device)
            d_logits = torch.empty((T, self.E), dtype=torch.float32, device=self.device)
        B.moe_combine_backward(self.desc(T), dy, y_rows, routing["topk_w"], routing["inv"], d_rows,
                               d_w, stream)
        B.moe_route_backward(self.route_desc(T), routing["logits"], routing["topk_idx"], d_w,
                             d_logits, stream)
        return {"d_y_rows": d_rows, "d_topk_w": d_w, "d_logits": d_logits}

    def stats(self, counts: torch.Tensor, T: int, straggler_mask: Optional[torch.Tensor] = None,
              stream=None) -> dict:
        return B.moe_expert_stats(self.desc(T), counts, straggler_mask, self.workspace(T), stream)

    def update_bias(self, counts: torch.Tensor, tokens: int, gamma: float, stream=None) -> None:
        """Dynamic bias update from expert counts accumulated over `tokens`
        tokens: B_e -= gamma for overloaded experts, += gamma for idle ones."""
        if self.tensors[5] is None:
            raise ValueError("the layer has no expert bias tensor to update")
        B.moe_bias_update(self.desc(tokens), counts, self.tensors[5], gamma, stream)


class MoEBlock:
    """h' = h + alpha * gate * u with u the MoE layer on rms(h) * w_pre, itself
    normalised by w_post where that is given.

    w_pre, w_post [H] and the per-channel gate [H] (or None) have the layer's dtype."""

    def __init__(self, layer: MoELayer, w_pre, w_post=None, gate=None, alpha: float = 1.0,
                 eps: float = 1e-6):
        self.layer = layer
        self.w_pre, self.w_post, self.gate = (t.contiguous() if t is not None else None
                                              for t in (w_pre, w_post, gate))
        self.alpha, self.eps = float(alpha), float(eps)

    def norm_desc(self, T: int, gate: str) -> B.MoENormDesc:
        return B.make_norm(T, self.layer.H, B.dtype_code(self.layer.dtype), gate=gate,
                           alpha=self.alpha, eps=self.eps)

    def pre_norm(self, h: torch.Tensor, stream=None) -> torch.Tensor:
        """rms(h) * w_pre, the input of the layer."""
        with _on(stream):
            x = torch.empty_like(h)
        B.moe_block_norm(self.norm_desc(h.shape[0], "none"), h, w_pre=self.w_pre, x=x,
                         stream=stream)
        return x

    def forward(self, h: torch.Tensor, x: Optional[torch.Tensor] = None, next_w_pre=None,
                routing: Optional[dict] = None, stream=None):
        """h' for the residual stream h [T, H]. `x`: the layer's input, if the block before
        has normalised it already. With next_w_pre [H] returns (h', rms(h') * next_w_pre):
        the residual, this block's post-norm and the next block's pre-norm in one pass."""
        with _on(stream):
            if x is None:
                x = self.pre_norm(h, stream)
            y = self.layer.forward(x, routing=routing, stream=stream)
            h_out = torch.empty_like(h)
            x_next = torch.empty_like(h) if next_w_pre is not None else None
        desc = self.norm_desc(h.shape[0], "none" if self.gate is None else "channel")
        B.moe_block_norm(desc, h, y, self.w_post, self.gate, next_w_pre, h_out, x_next, stream)
        return h_out if next_w_pre is None else (h_out, x_next)

    __call__ = forward


class DenseFFN:
    """Dense feed-forward y = act(x W1^T + b1) W2^T + b2 (+ residual), the dense layers
    beside the MoE ones. Weights w1 [D, H], w2 [H, D], biases b1 [D], b2 [H] or None,
    all of one dtype."""

    def __init__(self, w1, w2, b1=None, b2=None, act: str = "gelu"):
        self.D, self.H = w1.shape
        self.dtype, self.device, self.act = w1.dtype, w1.device, act
        self.w1, self.w2, self.b1, self.b2 = (t.contiguous() if t is not None else None
                                              for t in (w1, w2, b1, b2))
        self._ws = {}   # one workspace per stream

    def descs(self, T: int):
        code = B.dtype_code(self.dtype)
        return (B.make_linear(T, self.H, self.D, code, self.act),
                B.make_linear(T, self.D, self.H, code))

    def workspace(self, T: int) -> torch.Tensor:
        """Workspace of calls with T tokens on the current stream. Calls on different
        streams may run at the same time, so each stream has its own, which grows with
        the batch. A call that is being captured gets one of its own from the graph's
        memory, zeroed by the graph: replays run beside eager calls and other graphs."""
        need = max(B.moe_linear_workspace_size(d) for d in self.descs(T))
        capturing = torch.cuda.is_current_stream_capturing()
        stream = torch.cuda.current_stream(self.device).cuda_stream
        ws = None if capturing else self._ws.get(stream)
        if ws is None or ws.numel() < need:
            if not capturing:
                self._ws.pop(stream, None)
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            ws[:B.MOE_LINEAR_WS_HEAD].zero_()
            if not capturing:
                self._ws[stream] = ws
        return ws

    def saved_buffers(self, T: int) -> dict:
        """Buffers that a forward pass fills for `backward`."""
        return {k: torch.empty((T, self.D), dtype=self.dtype, device=self.device)
                for k in ("pre", "hidden")}

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                saved: Optional[dict] = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        first, second = self.descs(T)
        with _on(stream):
            hidden = saved["hidden"] if saved is not None else \
                torch.empty((T, self.D), dtype=self.dtype, device=self.device)
            y = torch.empty_like(x)
            ws = self.workspace(T)
        pre = saved["pre"] if saved is not None and self.act != "none" else None
        with _launching:
            B.moe_linear(first, x, self.w1, self.b1, None, pre, hidden, ws, stream)
            B.moe_linear(second, hidden, self.w2, self.b2, residual, None, y, ws, stream)
        return y

    __call__ = forward

    def backward(self, dy: torch.Tensor, x: torch.Tensor, saved: dict, stream=None) -> dict:
        """Gradients dx, dw1, dw2 (the weights' dtype), db1, db2 (fp32, where the layer
        has that bias). The residual's gradient is dy."""
        T = x.shape[0]
        first, second = self.descs(T)
        new = torch.empty_like

        def bias_grad(b):
            return torch.empty(b.shape, dtype=torch.float32, device=b.device) if b is not None else None

        with _on(stream):
            ws = self.workspace(T)
            out = {"dx": new(x), "dw1": new(self.w1), "dw2": new(self.w2), "db1": bias_grad(self.b1),
                   "db2": bias_grad(self.b2)}
            d_hidden = new(saved["hidden"])
        with _launching:
            B.moe_linear_backward(second, dy, saved["hidden"], self.w2, None, d_hidden, out["dw2"],
                                  out["db2"], ws, stream)
            B.moe_linear_backward(first, d_hidden, x, self.w1,
                                  saved["pre"] if self.act != "none" else None, out["dx"],
                                  out["dw1"], out["db1"], ws, stream)
        return {k: v for k, v in out.items() if v is not None}
