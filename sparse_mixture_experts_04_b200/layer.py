"""MoeLayer: one layer's weights, workspace and routing buffers on the device,
with forward() = one moe_layer_forward call, and forward_host() for batches
that live in (pinned) host memory.  Allocation (through torch), stream
bookkeeping and argument marshalling only."""
from __future__ import annotations

import torch

from . import api


class MoeLayer:
    # the C entry points behind the methods (MoeLayerI8 has its own)
    _alloc_workspace = staticmethod(api.alloc_workspace)
    _forward = staticmethod(api.moe_layer_forward)
    _forward_few = staticmethod(api.moe_layer_forward_few)

    def __init__(self, prob: api.MoeProblem, weights: dict, device="cuda", keep_routing: bool = True):
        self.prob = prob
        self.device = torch.device(device)
        self.weights = weights
        self.ws = self._alloc_workspace(prob, self.device)
        self.few_ws = None  # forward_few's workspace, allocated by its first call on that call's stream
        self._few_streams = set()  # handles of the streams that have used it
        self.dtype = torch.bfloat16 if prob.dtype == api.DTYPE_BF16 else torch.float32
        T, E, K = prob.T, prob.n_experts, prob.top_k
        self.routing = None
        if keep_routing:
            i32 = dict(dtype=torch.int32, device=self.device)
            self.routing = dict(
                logits=torch.empty((T, E), dtype=torch.float32, device=self.device),
                topk_idx=torch.empty((T, K), **i32), topk_w=torch.empty((T, K), dtype=torch.float32, device=self.device),
                counts=torch.empty(E, **i32), kept=torch.empty(E, **i32), seg_off=torch.empty(E + 1, **i32),
                slot_of=torch.empty((T, K), **i32), perm=torch.empty(max(api.max_rows(prob), 1), **i32))
        self.stats = torch.empty(api.stats_size(prob), dtype=torch.float32, device=self.device)
        if prob.flags & api.FLAG_EXPERT_CAPACITY and weights.get("expert_capacity") is None:
            # start from the uniform capacity (no limit: -1)
            cap = api.capacity(prob)
            cap = -1 if cap < 0 else min(cap, T)
            weights["expert_capacity"] = torch.full((E,), cap, dtype=torch.int32, device=self.device)
        self._balance_step = 0
        self._count_hist = None
        self._last = None  # whose call left the routing arrays: "forward" or "few"

    @classmethod
    def from_inputs(cls, inputs: dict, device="cuda", flags: int = 0, keep_routing: bool = True) -> "MoeLayer":
        """Build from synth.generate() output (CPU tensors are copied to the device)."""
        cfg = inputs["cfg"]
        prob = api.make_problem(cfg.T, cfg.d_model, cfg.n_experts, cfg.top_k, cfg.d_ff, cfg.n_shared,
                                cfg.capacity_factor, cfg.dtype, flags, cfg.alpha)
        dev = torch.device(device)

        def to_dev(v):
            if v is None:
                return None
            t = torch.as_tensor(v)
            return t.to(dev).contiguous()

        w = {k: to_dev(inputs.get(k)) for k in ("w_gate", "w13", "w2", "w13_shared", "w2_shared")}
        w["sel_bias"] = to_dev(inputs.get("sel_bias"))
        w["logit_offset"] = to_dev(inputs.get("logit_offset"))
        return cls(prob, w, dev, keep_routing)

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, with_stats: bool = True,
                stream=None) -> torch.Tensor:
        if y is None:
            y = api._empty((self.prob.T, self.prob.d_model), self.dtype, self.device, stream)
        self._forward(self.prob, x, self.weights, y, self.routing, self.stats if with_stats else None, self.ws, stream)
        self._last = "forward"
        return y

    __call__ = forward

    def forward_few(self, x: torch.Tensor, y: torch.Tensor | None = None, with_stats: bool = True,
                    stream=None) -> torch.Tensor:
        """forward() in one kernel, for layers of at most api.FEW_MAX_TOKENS
        tokens (decode steps): same inputs, outputs, routing and statistics.
        Agrees with forward() to rounding (hidden activations and expert
        outputs keep more bits up to the combine).  Up to twice as fast for
        one token; from 32 tokens on forward() can be the faster.

        No backward() from it: that reads what forward() leaves behind, and the
        routing arrays (self.routing) belong to both.  backward() refuses until
        the next forward(); a replayed graph of this call overwrites them unseen,
        so replay none between forward() and backward().  A layer built with
        keep_routing=False has no such arrays, and a pending backward() stays
        good.  Its device status is in self.few_ws."""
        dev = api._cuda("x", x)
        if y is None:
            y = api._empty((self.prob.T, self.prob.d_model), self.dtype, self.device, stream)
        handle = api._stream_handle(stream, dev)
        if self.few_ws is None:
            self._check_weights()
            with api._on_stream(stream, dev):  # its clearing runs in front of the kernel, on the same stream
                self.few_ws = api.alloc_few_workspace(self.prob, self.device)
            self._few_streams = {handle}
        elif handle not in self._few_streams:  # freed while this stream still uses it, it is not handed out again
            with api._on_stream(stream, dev):
                self.few_ws.record_stream(torch.cuda.current_stream(dev))
            self._few_streams.add(handle)
        self._forward_few(self.prob, x, self.weights, y, self.routing, self.stats if with_stats else None,
                          self.few_ws, handle)
        if self.routing is not None or self._last is None:
            self._last = "few"
        return y

    def _weight_shapes(self) -> dict:
        """Expected (shape, dtype) of the weights a forward reads."""
        P = self.prob
        E, d, F, Ns = P.n_experts, P.d_model, P.d_ff, P.n_shared
        out = {"w13": ((E, 2 * F, d), self.dtype), "w2": ((E, d, F), self.dtype)}
        if not P.flags & api.FLAG_LOGITS_GIVEN:
            out["w_gate"] = ((E, d), self.dtype)
        if Ns:
            out.update(w13_shared=((Ns, 2 * F, d), self.dtype), w2_shared=((Ns, d, F), self.dtype))
        return out

    def _check_weights(self) -> None:
        """Raise ValueError unless the weights have the problem's shapes and types and
        are on the layer's device."""
        E = self.prob.n_experts
        for name, (shape, dtype) in self._weight_shapes().items():
            t = self.weights.get(name)
            if (t is None or tuple(t.shape) != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or
                    t.device != self.ws.device):
                raise ValueError(f"weights['{name}'] must be a contiguous CUDA {dtype} tensor of shape {shape} on the "
                                 "layer's device")
        for name, dtype in (("logit_offset", torch.float32), ("sel_bias", torch.float32),
                            ("expert_capacity", torch.int32)):
            t = self.weights.get(name)
            if t is not None and (tuple(t.shape) != (E,) or t.dtype != dtype or not t.is_cuda or
                                  not t.is_contiguous() or t.device != self.ws.device):
                raise ValueError(f"weights['{name}'] must be a contiguous CUDA {dtype} tensor of shape {(E,)} on the "
                                 "layer's device")

    def capture(self, with_stats: bool = True) -> None:
        """Capture one forward into a CUDA graph over static input/output
        buffers (self.graph_x, self.graph_y); forward_graphed() replays it.  The
        layer's launches (memset, kernels with programmatic dependent launch)
        become one graph, so a replay costs one launch on the host.  One eager
        forward runs first, outside the capture, to set the kernels' per-device
        attributes."""
        T, d = self.prob.T, self.prob.d_model
        self.graph_x = torch.zeros((T, d), dtype=self.dtype, device=self.device)
        self.graph_y = torch.empty((T, d), dtype=self.dtype, device=self.device)
        self.forward(self.graph_x, self.graph_y, with_stats)
        torch.cuda.synchronize(self.device)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self._forward(self.prob, self.graph_x, self.weights, self.graph_y, self.routing,
                          self.stats if with_stats else None, self.ws)
        self._graph = g

    def forward_graphed(self, x: torch.Tensor | None = None) -> torch.Tensor:
        """Replay the captured forward (capture() first) on the current stream;
        x (if given) is copied into the static input first.  Returns the static
        output buffer, overwritten by the next replay."""
        if getattr(self, "_graph", None) is None:
            raise RuntimeError("MoeLayer.capture() has not been called")
        if x is not None:
            self.graph_x.copy_(x)
        self._graph.replay()
        self._last = "forward"
        return self.graph_y

    def backward(self, x: torch.Tensor, dy: torch.Tensor, d_loss: float = 1.0, d_zloss: float = 0.0,
                 stream=None) -> dict:
        """Gradients of the last forward (same x; the workspace and the routing
        arrays untouched since), for dJ/dy = dy and dJ/d(balance loss) = d_loss,
        dJ/d(z-loss) = d_zloss.  Returns FP32 weight gradients and dx (activation
        dtype).  RuntimeError after forward_few(), which overwrites the routing."""
        if self._last == "few":
            raise RuntimeError("backward() needs a forward() of the same x: forward_few() was the last call, and it "
                               "leaves no activations and another routing")
        P, dev = self.prob, self.device
        f32 = dict(dtype=torch.float32, device=dev)
        E, d, F, Ns, T = P.n_experts, P.d_model, P.d_ff, P.n_shared, P.T
        g = dict(dx=torch.empty((T, d), dtype=self.dtype, device=dev), dw13=torch.empty((E, 2 * F, d), **f32),
                 dw2=torch.empty((E, d, F), **f32), d_offset=torch.empty(E, **f32),
                 d_logits=torch.empty((T, E), **f32))
        if not P.flags & api.FLAG_LOGITS_GIVEN:
            g["dw_gate"] = torch.empty((E, d), **f32)
        if Ns:
            g["dw13_shared"] = torch.empty((Ns, 2 * F, d), **f32)
            g["dw2_shared"] = torch.empty((Ns, d, F), **f32)
        if getattr(self, "_bwd_ws", None) is None:
            with api._on_stream(stream, dev.index):  # its clearing runs in front of the kernels
                self._bwd_ws = api.alloc_backward_workspace(P, dev)
        api.moe_layer_backward(P, x, self.weights, self.routing, self.ws, dy, d_loss, d_zloss, g, self._bwd_ws,
                               stream)
        return g

    def balance_update(self, bias_rate: float = 0.0, bias_mode: int = api.BIAS_UPDATE_SIGN, c_base: float | None = None,
                       gamma: float = 0.0, window: int = 8, stream=None) -> None:
        """Between steps: move the selection bias against the last forward's
        load (when the layer has one and bias_rate != 0) and, for a layer built
        with FLAG_EXPERT_CAPACITY, set the next forward's per-expert capacities
        from the last `window` forwards' loads (c_base defaults to the
        problem's capacity factor).  One kernel on the stream."""
        if self.routing is None:
            raise ValueError("balance_update needs the routing outputs (keep_routing=True)")
        bias = self.weights.get("sel_bias") if bias_rate != 0.0 else None
        caps = self.weights.get("expert_capacity") if self.prob.flags & api.FLAG_EXPERT_CAPACITY else None
        if bias is None and caps is None:
            return
        hist = None
        if caps is not None:
            if self._count_hist is None or self._count_hist.shape[0] != window:
                with api._on_stream(stream, self.device.index):
                    self._count_hist = torch.zeros((window, self.prob.n_experts), dtype=torch.int32, device=self.device)
                self._balance_step = 0
            hist = self._count_hist
        cb = self.prob.capacity_factor if c_base is None else c_base
        api.moe_balance_update(self.prob, self.routing["counts"], bias, bias_rate, bias_mode, hist,
                               self._balance_step, cb, gamma, caps, stream)
        if caps is not None:
            self._balance_step += 1

    def forward_host(self, xs_host, ys_host, stats_host=None, stream=None):
        """Run one layer forward per host batch: xs_host[i] [T, d] -> ys_host[i].

        Host tensors should be pinned.  The host->device copy of batch i+1 and
        the device->host copy of batch i-1 run on their own streams while batch
        i computes (two device buffers each for x and y), so the copy engines
        overlap the kernels.  stats_host[i] (optional) receives the [2E+1]
        statistics of batch i.  Returns after every copy has landed."""
        n = len(xs_host)
        if n == 0:
            return
        dev = self.device
        comp = stream if stream is not None else torch.cuda.current_stream(dev)
        h2d, d2h = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
        T, d = self.prob.T, self.prob.d_model
        xb = [torch.empty((T, d), dtype=self.dtype, device=dev) for _ in range(2)]
        yb = [torch.empty((T, d), dtype=self.dtype, device=dev) for _ in range(2)]
        sb = [torch.empty_like(self.stats) for _ in range(2)]
        ev = lambda: torch.cuda.Event()
        copied_in = [ev() for _ in range(n)]
        computed = [ev() for _ in range(n)]
        copied_out = [ev() for _ in range(n)]
        h2d.wait_stream(comp)
        d2h.wait_stream(comp)
        for i in range(n):
            b = i % 2
            with torch.cuda.stream(h2d):
                if i >= 2:
                    h2d.wait_event(computed[i - 2])       # x buffer b is free again
                xb[b].copy_(xs_host[i], non_blocking=True)
                copied_in[i].record(h2d)
            comp.wait_event(copied_in[i])
            if i >= 2:
                comp.wait_event(copied_out[i - 2])        # y / stats buffers b are free again
            self._forward(self.prob, xb[b], self.weights, yb[b], self.routing, sb[b], self.ws, comp)
            computed[i].record(comp)
            with torch.cuda.stream(d2h):
                d2h.wait_event(computed[i])
                ys_host[i].copy_(yb[b], non_blocking=True)
                if stats_host is not None:
                    stats_host[i].copy_(sb[b], non_blocking=True)
                copied_out[i].record(d2h)
        self._last = "forward"
        comp.wait_stream(d2h)
        comp.synchronize()


def quantize_weights(weights: dict) -> dict:
    """The weights of a layer (w13, w2 and the shared ones, BF16 or FP32, on a
    CUDA device) to 8 bits with a scale per output channel, for MoeLayerI8.
    w_gate and logit_offset are passed on; sel_bias and expert_capacity, which
    balance_update() writes, are copied.  The shared experts are
    one expert of width N_s * F: w2_shared has one scale per output channel
    over all of them."""
    out = {k: weights.get(k) for k in ("w_gate", "logit_offset")}
    for k in ("sel_bias", "expert_capacity"):
        out[k] = None if weights.get(k) is None else weights[k].clone()
    for k in ("w13", "w2", "w13_shared"):
        if weights.get(k) is not None:
            out[k], out[k + "_scale"] = api.quantize_rows(weights[k])
    w2s = weights.get("w2_shared")
    if w2s is not None:
        n, d, F = w2s.shape
        q, out["w2_shared_scale"] = api.quantize_rows(w2s.permute(1, 0, 2).reshape(d, n * F).contiguous())
        out["w2_shared"] = q.view(d, n, F).permute(1, 0, 2).contiguous()
    return out


class MoeLayerI8(MoeLayer):
    """MoeLayer with 8-bit experts: the same forward(), forward_few(), capture()
    and balance_update() over weights from quantize_weights (or the caller's
    own int8 matrices and scales; see moe_weights_i8_t in the header).  Token
    rows and hidden rows are quantised on the way.  BF16 activations, d_model
    and d_ff multiples of 16.  Inference only."""
    _alloc_workspace = staticmethod(api.alloc_i8_workspace)
    _forward = staticmethod(api.moe_layer_forward_i8)
    _forward_few = staticmethod(api.moe_layer_forward_few_i8)

    def __init__(self, prob: api.MoeProblem, weights: dict, device="cuda", keep_routing: bool = True):
        super().__init__(prob, weights, device, keep_routing)
        self._check_weights()

    def _weight_shapes(self) -> dict:
        P = self.prob
        E, d, F, Ns = P.n_experts, P.d_model, P.d_ff, P.n_shared
        i8, f32 = torch.int8, torch.float32
        out = {"w13": ((E, 2 * F, d), i8), "w13_scale": ((E, 2 * F), f32), "w2": ((E, d, F), i8),
               "w2_scale": ((E, d), f32)}
        if not P.flags & api.FLAG_LOGITS_GIVEN:
            out["w_gate"] = ((E, d), self.dtype)
        if Ns:
            out.update(w13_shared=((Ns, 2 * F, d), i8), w13_shared_scale=((Ns, 2 * F), f32),
                       w2_shared=((Ns, d, F), i8), w2_shared_scale=((d,), f32))
        return out

    @classmethod
    def from_layer(cls, layer: MoeLayer, keep_routing: bool = True) -> "MoeLayerI8":
        """Quantise an existing layer's weights.  The layer keeps its own; both
        adapt apart from each other (balance_update), from the same start.
        FLAG_SAVE_GU, which serves the backward, is dropped."""
        prob = type(layer.prob).from_buffer_copy(layer.prob)
        prob.flags &= ~api.FLAG_SAVE_GU
        return cls(prob, quantize_weights(layer.weights), layer.device, keep_routing)

    @classmethod
    def from_inputs(cls, inputs: dict, device="cuda", flags: int = 0, keep_routing: bool = True) -> "MoeLayerI8":
        return cls.from_layer(MoeLayer.from_inputs(inputs, device, flags, False), keep_routing)

    def backward(self, *args, **kwargs):
        raise RuntimeError("8-bit experts have no backward: train with MoeLayer and quantise its weights")
